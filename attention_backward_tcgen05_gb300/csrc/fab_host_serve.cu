// fab_host_serve.cu -- the C ABI of the operators around the attention
// (declared in include/fab.h): query/key norms with the position rotation and
// their gradient, appending to a paged key/value cache, attention over it.
// Argument validation and launches only; nothing allocates or synchronises.
#include <math.h>

#include "fab.h"
#include "fab_internal.h"

#define FAB_API extern "C" FAB_EXPORT

namespace fab {
namespace {

constexpr int64_t kMaxInt32 = 2147483647;
// Tokens of a paged call: the attention kernels number those of its last unit in 32
// bits up to the end of the unit's tiles, 255 past the last that is there.
constexpr int64_t kMaxTokens = kMaxInt32 - 256;

int64_t elem_size(int dtype) { return dtype == FAB_F32 ? 4 : 2; }

bool aligned(const void* p, int64_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % (uintptr_t)a == 0; }

// a * b * c * d <= kMaxElems for positive factors
bool fits(int64_t a, int64_t b, int64_t c, int64_t d) {
  return a <= kMaxElems / b && a * b <= kMaxElems / c && a * b * c <= kMaxElems / d;
}

bool heads_ok(int64_t H, int64_t Hkv, int64_t DK, int64_t DV) {
  return H > 0 && H <= kMaxInt32 && Hkv > 0 && DK > 0 && DV > 0 && H % Hkv == 0;
}

bool rot_ok(int64_t rot, int64_t DK, int64_t P) {
  return rot >= 0 && rot <= DK && rot % 2 == 0 && (rot == 0 || (P > 0 && P <= kMaxInt32));
}

// `rows` rows of `heads` heads of `width` columns, `ld` elements apart
bool rows_ok(int64_t rows, int64_t heads, int64_t width, int64_t ld) {
  return fits(rows, heads, width, 1) && ld >= heads * width && ld <= kMaxElems / rows;
}

int check_rope_dims(const fab_rope_dims* d) {
  if (!d || d->B <= 0 || d->N <= 0 || !heads_ok(d->H, d->Hkv, d->DK, d->DV)) return FAB_ERR_INVALID;
  if (!rot_ok(d->rot, d->DK, d->P)) return FAB_ERR_INVALID;
  if (!fits(d->B, d->N, d->H, d->DK) || !fits(d->B, d->N, d->Hkv, d->DV)) return FAB_ERR_INVALID;
  return FAB_OK;
}

int check_paged_dims(const fab_paged_dims* d) {
  if (!d || d->B <= 0 || d->T < 0 || !heads_ok(d->H, d->Hkv, d->DK, d->DV)) return FAB_ERR_INVALID;
  if (d->page <= 0 || d->pages <= 0 || d->max_pages <= 0) return FAB_ERR_INVALID;
  if (d->B >= kMaxInt32 || d->T > kMaxTokens || d->page > kMaxInt32 || d->pages > kMaxInt32 || d->max_pages > kMaxInt32)
    return FAB_ERR_INVALID;
  if (!fits(d->pages, d->page, d->Hkv, d->DK) || !fits(d->pages, d->page, d->Hkv, d->DV)) return FAB_ERR_INVALID;
  if (!fits(d->B, d->max_pages, 1, 1)) return FAB_ERR_INVALID;
  if (d->T > 0 && (!fits(d->T, d->H, d->DK, 1) || !fits(d->T, d->H, d->DV, 1))) return FAB_ERR_INVALID;
  return FAB_OK;
}

bool widths_ok(int64_t DK, int64_t DV) { return DK <= kMaxWidth && DV <= kMaxWidth; }

// What the norm and the rotation read besides the rows: optional weights,
// tables, eps.
int check_norm_rope(int dtype, const void* wq, const void* wk, const float* cos, const float* sin, int64_t rot,
                    float eps) {
  if (!dtype_ok(dtype)) return FAB_ERR_INVALID;
  const int64_t e = elem_size(dtype);
  if ((wq && !aligned(wq, e)) || (wk && !aligned(wk, e))) return FAB_ERR_INVALID;
  if (rot > 0 && (!aligned(cos, 4) || !aligned(sin, 4))) return FAB_ERR_INVALID;
  if (!(eps >= 0.f) || isinf(eps)) return FAB_ERR_INVALID;
  return FAB_OK;
}

RopeProblem rope_problem(const fab_rope_dims* d, int dtype, float eps, int interleaved) {
  RopeProblem p{};
  p.B = d->B;
  p.N = d->N;
  p.H = d->H;
  p.Hkv = d->Hkv;
  p.DK = d->DK;
  p.DV = d->DV;
  p.rot = d->rot;
  p.P = d->P;
  p.ldq = d->ldq;
  p.ldk = d->ldk;
  p.ldv = d->ldv;
  p.ldgq = d->ldgq;
  p.ldgk = d->ldgk;
  p.ldgv = d->ldgv;
  p.eps = eps;
  p.interleaved = interleaved ? 1 : 0;
  p.dtype = dtype;
  return p;
}

PagedProblem paged_problem(const fab_paged_dims* d, int dtype) {
  PagedProblem p{};
  p.B = d->B;
  p.T = d->T;
  p.H = d->H;
  p.Hkv = d->Hkv;
  p.DK = d->DK;
  p.DV = d->DV;
  p.page = d->page;
  p.pages = d->pages;
  p.max_pages = d->max_pages;
  p.dtype = dtype;
  return p;
}

size_t paged_workspace_bytes(const PagedProblem& p) {
  return paged_tc_supported(p) ? paged_tc_workspace_bytes(p) : paged_simt_workspace_bytes(p);
}

}  // namespace
}  // namespace fab

using namespace fab;

FAB_API int fab_qk_norm_rope(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                             const float* cos, const float* sin, const int32_t* pos, float eps, int interleaved,
                             int dtype, const fab_rope_dims* dims, void* q_out, void* k_out, void* v_out,
                             fab_stream stream) {
  int rc = check_rope_dims(dims);
  if (rc != FAB_OK) return rc;
  rc = check_norm_rope(dtype, wq, wk, cos, sin, dims->rot, eps);
  if (rc != FAB_OK) return rc;
  const int64_t e = elem_size(dtype), rows = dims->B * dims->N;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, 16) || !aligned(k_out, 16)) return FAB_ERR_INVALID;
  if ((v == nullptr) != (v_out == nullptr)) return FAB_ERR_INVALID;
  if (v && (!aligned(v, e) || !aligned(v_out, 16))) return FAB_ERR_INVALID;
  if (!rows_ok(rows, dims->H, dims->DK, dims->ldq) || !rows_ok(rows, dims->Hkv, dims->DK, dims->ldk))
    return FAB_ERR_INVALID;
  if (v && !rows_ok(rows, dims->Hkv, dims->DV, dims->ldv)) return FAB_ERR_INVALID;
  if (dims->rot > 0 && ((pos && !aligned(pos, 4)) || (!pos && dims->N > dims->P))) return FAB_ERR_INVALID;
  if (!widths_ok(dims->DK, dims->DV)) return FAB_ERR_UNSUPPORTED;
  RopeProblem p = rope_problem(dims, dtype, eps, interleaved);
  p.q = q;
  p.k = k;
  p.v = v;
  p.wq = wq;
  p.wk = wk;
  p.cos = cos;
  p.sin = sin;
  p.pos = pos;
  p.q_out = q_out;
  p.k_out = k_out;
  p.v_out = v_out;
  return from_cuda(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

FAB_API size_t fab_qk_norm_rope_backward_workspace_bytes(const fab_rope_dims* dims) {
  if (check_rope_dims(dims) != FAB_OK) return 0;
  return (size_t)(kRopePartialRows * dims->DK) * sizeof(float);
}

FAB_API int fab_qk_norm_rope_backward(const float* dq, const float* dk, const float* dv, const void* q, const void* k,
                                      const void* wq, const void* wk, const float* cos, const float* sin,
                                      const int32_t* pos, float eps, int interleaved, int dtype,
                                      const fab_rope_dims* dims, void* workspace, size_t workspace_bytes, void* gq,
                                      void* gk, void* gv, float* gwq, float* gwk, fab_stream stream) {
  int rc = check_rope_dims(dims);
  if (rc != FAB_OK) return rc;
  rc = check_norm_rope(dtype, wq, wk, cos, sin, dims->rot, eps);
  if (rc != FAB_OK) return rc;
  const int64_t e = elem_size(dtype), rows = dims->B * dims->N;
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(gq, e) || !aligned(gk, e)) return FAB_ERR_INVALID;
  if ((dv == nullptr) != (gv == nullptr)) return FAB_ERR_INVALID;
  if (dv && (!aligned(dv, 16) || !aligned(gv, e))) return FAB_ERR_INVALID;
  if ((wq == nullptr) != (gwq == nullptr) || (wk == nullptr) != (gwk == nullptr)) return FAB_ERR_INVALID;
  if ((gwq && !aligned(gwq, 16)) || (gwk && !aligned(gwk, 16))) return FAB_ERR_INVALID;
  if (wq && (!aligned(q, e) || !rows_ok(rows, dims->H, dims->DK, dims->ldq))) return FAB_ERR_INVALID;
  if (wk && (!aligned(k, e) || !rows_ok(rows, dims->Hkv, dims->DK, dims->ldk))) return FAB_ERR_INVALID;
  if (!rows_ok(rows, dims->H, dims->DK, dims->ldgq) || !rows_ok(rows, dims->Hkv, dims->DK, dims->ldgk))
    return FAB_ERR_INVALID;
  if (dv && !rows_ok(rows, dims->Hkv, dims->DV, dims->ldgv)) return FAB_ERR_INVALID;
  if (dims->rot > 0 && ((pos && !aligned(pos, 4)) || (!pos && dims->N > dims->P))) return FAB_ERR_INVALID;
  if ((wq || wk) &&
      (!aligned(workspace, 16) || workspace_bytes < fab_qk_norm_rope_backward_workspace_bytes(dims)))
    return FAB_ERR_WORKSPACE;
  if (!widths_ok(dims->DK, dims->DV)) return FAB_ERR_UNSUPPORTED;
  RopeProblem p = rope_problem(dims, dtype, eps, interleaved);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.q = q;
  p.k = k;
  p.wq = wq;
  p.wk = wk;
  p.cos = cos;
  p.sin = sin;
  p.pos = pos;
  p.gq = gq;
  p.gk = gk;
  p.gv = gv;
  p.gwq = gwq;
  p.gwk = gwk;
  p.partial = static_cast<float*>(workspace);
  return from_cuda(launch_rope_backward(p, static_cast<cudaStream_t>(stream)));
}

FAB_API int fab_paged_append(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                             const float* cos, const float* sin, float eps, int interleaved, const int32_t* starts,
                             const int32_t* lens, const int32_t* table, int dtype, const fab_paged_dims* dims,
                             void* q_out, void* k_cache, void* v_cache, fab_stream stream) {
  int rc = check_paged_dims(dims);
  if (rc != FAB_OK) return rc;
  if (!rot_ok(dims->rot, dims->DK, dims->P)) return FAB_ERR_INVALID;
  rc = check_norm_rope(dtype, wq, wk, cos, sin, dims->rot, eps);
  if (rc != FAB_OK) return rc;
  if (!aligned(starts, 4) || !aligned(lens, 4) || !aligned(table, 4)) return FAB_ERR_INVALID;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return FAB_ERR_INVALID;
  if (!widths_ok(dims->DK, dims->DV)) return FAB_ERR_UNSUPPORTED;
  if (dims->T == 0) return FAB_OK;
  const int64_t e = elem_size(dtype);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(q_out, 16)) return FAB_ERR_INVALID;
  if (!rows_ok(dims->T, dims->H, dims->DK, dims->ldq) || !rows_ok(dims->T, dims->Hkv, dims->DK, dims->ldk) ||
      !rows_ok(dims->T, dims->Hkv, dims->DV, dims->ldv))
    return FAB_ERR_INVALID;
  RopeProblem p{};
  p.B = 1;
  p.N = dims->T;
  p.H = dims->H;
  p.Hkv = dims->Hkv;
  p.DK = dims->DK;
  p.DV = dims->DV;
  p.rot = dims->rot;
  p.P = dims->P;
  p.ldq = dims->ldq;
  p.ldk = dims->ldk;
  p.ldv = dims->ldv;
  p.eps = eps;
  p.interleaved = interleaved ? 1 : 0;
  p.dtype = dtype;
  p.q = q;
  p.k = k;
  p.v = v;
  p.wq = wq;
  p.wk = wk;
  p.cos = cos;
  p.sin = sin;
  p.starts = starts;
  p.lens = lens;
  p.table = table;
  p.seqs = dims->B;
  p.page = dims->page;
  p.pages = dims->pages;
  p.max_pages = dims->max_pages;
  p.q_out = q_out;
  p.k_out = k_cache;
  p.v_out = v_cache;
  return from_cuda(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

FAB_API size_t fab_paged_attention_workspace_bytes(const fab_paged_dims* dims, int dtype) {
  if (check_paged_dims(dims) != FAB_OK || !dtype_ok(dtype)) return 0;
  return paged_workspace_bytes(paged_problem(dims, dtype));
}

FAB_API int fab_paged_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* starts,
                                const int32_t* lens, const int32_t* table, int causal, float scale, int dtype,
                                const fab_paged_dims* dims, void* workspace, size_t workspace_bytes, void* o,
                                float* lse, fab_stream stream) {
  const int rc = check_paged_dims(dims);
  if (rc != FAB_OK) return rc;
  if (!dtype_ok(dtype) || !isfinite(scale)) return FAB_ERR_INVALID;
  if (!aligned(starts, 4) || !aligned(lens, 4) || !aligned(table, 4)) return FAB_ERR_INVALID;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return FAB_ERR_INVALID;
  if (dims->T > 0 && (!aligned(q, 16) || !aligned(o, 16) || (lse && !aligned(lse, 16)))) return FAB_ERR_INVALID;
  if (!widths_ok(dims->DK, dims->DV)) return FAB_ERR_UNSUPPORTED;
  if (dims->T == 0) return FAB_OK;
  PagedProblem p = paged_problem(dims, dtype);
  const size_t need = paged_workspace_bytes(p);
  if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return FAB_ERR_WORKSPACE;
  p.scale = scale;
  p.causal = causal ? 1 : 0;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.starts = starts;
  p.lens = lens;
  p.table = table;
  p.o = o;
  p.lse = lse;
  p.workspace = workspace;
  if (paged_tc_supported(p)) {
    if (!encode_tiled_fn()) return FAB_ERR_CUDA;
    return from_cuda(launch_paged_tc(p, static_cast<cudaStream_t>(stream)));
  }
  return from_cuda(launch_paged_simt(p, static_cast<cudaStream_t>(stream)));
}
