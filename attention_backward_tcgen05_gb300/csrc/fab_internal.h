// fab_internal.h -- declarations shared by the host layer and the kernel
// translation units of libfab.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fab {

// Error bits a kernel may OR into its translation unit's device error word.
constexpr uint32_t kErrTimeout = 1u;
constexpr uint32_t kErrSmemAlign = 2u;  // dynamic shared memory not 1024-byte aligned
constexpr uint32_t kErrIndex = 4u;      // a position, page or start read from device memory is out of range

// One validated call, in the units the kernels use.
struct Problem {
  int64_t B, H, Hkv, N, M, DK, DV;
  float scale;
  int causal;
  int dtype;  // FAB_F32, FAB_BF16 or FAB_F16
  const void* q;
  const void* k;
  const void* v;
  const void* d;  // upstream gradient, [DV,H,N,B]
  const void* o;  // forward output, [DV,H,N,B]
  const float* lse;
  const uint16_t* mask;  // f16 [M,N] or null
  float* di;             // workspace: D_i, f32 [N,H,B]
  // workspace, only with a mask: one byte per 128 x 128 tile of the mask,
  // nonzero when the tile holds an entry other than -inf, stored twice:
  // kt_live has a row per query tile over the key tiles, qt_live (right
  // after it) a row per key tile over the query tiles, each row
  // live_stride(tiles) bytes.  A pass skips the tiles before the first and
  // after the last live tile of its row.  Null: no skipping.
  uint8_t* kt_live;
  uint8_t* qt_live;
  float* packed;         // packed f32 result
  size_t off_k, off_v, end;  // bytes
};

// fab_preprocess.cu: D_i = rowsum(dO * O) into p.di; zero the padding of the
// packed result.
cudaError_t launch_preprocess(const Problem& p, cudaStream_t s);

// Bytes per row of a live-tile map over `tiles` tiles: padded to 16 so that
// rows can be read in 16-byte pieces.
__host__ __device__ inline int64_t live_stride(int64_t tiles) { return (tiles + 15) / 16 * 16; }

// fab_preprocess.cu: p.kt_live and p.qt_live from the mask (both non-null).
cudaError_t launch_mask_scan(const Problem& p, cudaStream_t s);

// fab_simt.cu: CUDA-core kernels for every dtype and width (DK, DV <= 256).
cudaError_t launch_forward_simt(const Problem& p, void* o, float* lse, cudaStream_t s);
cudaError_t launch_backward_simt(const Problem& p, cudaStream_t s);

// fab_fwd_tc.cu: the tcgen05 tensor-core forward with LSE (bf16 or f16, DK == DV in {64, 128}).
bool forward_tc_supported(const Problem& p);
cudaError_t launch_forward_tc(const Problem& p, void* o, float* lse, cudaStream_t s);

// fab_bwd_tc.cu: the tcgen05 tensor-core backward's key/value pass (dK, dV;
// bf16 or f16, DK == DV in {64, 128}).
bool backward_tc_supported(const Problem& p);
cudaError_t launch_backward_tc(const Problem& p, cudaStream_t s);

// fab_dq_tc.cu: the tcgen05 tensor-core backward's query pass (dQ), same
// problems as launch_backward_tc.  With fuse_d it also computes D_i from p.o
// into p.di and zeroes the packed result's padding (the preprocess's work);
// otherwise it reads D_i from p.di.
cudaError_t launch_dq_tc(const Problem& p, bool fuse_d, cudaStream_t s);

// One validated call of the norm + rotation entry points (fab_rope.cu).
struct RopeProblem {
  int64_t B, N, H, Hkv, DK, DV, rot, P;
  int64_t ldq, ldk, ldv, ldgq, ldgk, ldgv;
  float eps;
  int interleaved;
  int dtype;
  const void *q, *k, *v;
  const void *wq, *wk;  // null: no norm
  const float *cos, *sin;
  const int32_t* pos;  // [N,B] or null: token n is at position n
  void *q_out, *k_out, *v_out;
  // appending to a paged cache (starts non-null; then B = 1, N = T): k_out and
  // v_out are the caches
  const int32_t *starts, *lens, *table;
  int64_t seqs, page, pages, max_pages;
  // appending drafted tokens (or null): row t of `words` words says which new
  // tokens of its sequence token t sees; it is rotated by its place on its path
  const uint32_t* seen;
  int64_t words;
  // backward
  const float *dq, *dk, *dv;
  void *gq, *gk, *gv;
  float *gwq, *gwk;
  float* partial;  // workspace: kRopePartialRows rows of DK floats
};
// Rows of partial sums of a backward call (q's and k's together at most).
constexpr int64_t kRopePartialRows = 1280;
cudaError_t launch_rope(const RopeProblem& p, cudaStream_t s);
cudaError_t launch_rope_backward(const RopeProblem& p, cudaStream_t s);

// One validated fab_paged_attention call.
struct PagedProblem {
  int64_t B, T, H, Hkv, DK, DV, page, pages, max_pages;
  float scale;
  int causal;
  int dtype;
  const void *q, *k, *v;
  const int32_t *starts, *lens, *table;
  const uint32_t* seen;  // drafted trees (then causal): [words,T], else null
  int64_t words;
  void* o;
  float* lse;  // or null
  void* workspace;
};
// fab_paged_tc.cu: tcgen05, bf16 or f16, DK and DV multiples of 8 up to 128,
// pages of a multiple of 8 rows.
bool paged_tc_supported(const PagedProblem& p);
size_t paged_tc_workspace_bytes(const PagedProblem& p);
cudaError_t launch_paged_tc(const PagedProblem& p, cudaStream_t s);
// fab_paged_simt.cu: CUDA cores, every dtype, DK, DV <= 256, any page.
size_t paged_simt_workspace_bytes(const PagedProblem& p);
cudaError_t launch_paged_simt(const PagedProblem& p, cudaStream_t s);

// fab_pages.cu: who sees whom in drafted trees, keeping an accepted path, and
// the pages of a cache.
struct CacheProblem {
  int64_t B, T, words, Hkv, DK, DV, page, pages, max_pages, layers, ldk, ldv;
  int dtype;
  const int32_t *starts, *lens;
  const uint32_t* seen;
  const int32_t* last;                // accept
  int32_t* lens_out;                  // accept
  int32_t *table, *refs, *spare;      // (accept reads the table only)
  const int32_t *kept, *source;       // reserve; source may be null
  void *k, *v;
  void* workspace;
};
cudaError_t launch_draft_tree(const int32_t* starts, const int32_t* parents, int64_t B, int64_t T, int64_t words,
                              uint32_t* seen, cudaStream_t s);
cudaError_t launch_paged_accept(const CacheProblem& p, cudaStream_t s);
size_t paged_reserve_workspace_bytes(const CacheProblem& p);
cudaError_t launch_paged_reserve(const CacheProblem& p, cudaStream_t s);

// fab_host.cu: the checks the entry points share.
bool dtype_ok(int dtype);
int from_cuda(cudaError_t e);
constexpr int64_t kMaxWidth = 256;  // DK, DV limit of every kernel
constexpr int64_t kMaxElems = int64_t(1) << 40;

// fab_host.cu: cuTensorMapEncodeTiled from the driver, looked up once.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

// Each kernel translation unit keeps a device error word; these read and
// clear it (host side, synchronous).
uint32_t take_error_tc();
uint32_t take_error_dq();
uint32_t take_error_fwd();
uint32_t take_error_rope();
uint32_t take_error_paged();
uint32_t take_error_paged_tc();
uint32_t take_error_pages();

}  // namespace fab
