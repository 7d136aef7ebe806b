// The calls of the gated linear recurrence over whole sequences, and the last step of dlam (the kernels:
// ssd_glr_forward.cu, ssd_glr_backward.cu).
#include <initializer_list>

#include "glr_common.cuh"

namespace ssd {
namespace glr {
namespace {

// dlam = s(lam) / softplus(lam) sum of n rows of part; the factor goes to 1 where both vanish.
__global__ void __launch_bounds__(1024) k_glr_lam(const float* __restrict__ part, int n, int D, const float* lam, float* dlam) {
  __shared__ float s[32][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += blockDim.y) v += part[(size_t)i * D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D) return;
  for (int i = 1; i < blockDim.y; ++i) v += s[i][threadIdx.x];
  const float l = lam[c];
  dlam[c] = v * (l < -60.f ? 1.f : sigmoid_f(l) / softplus_f(l));
}

long long mark_count(const Args& a) { return (long long)axes(a) * ((a.T + mark_of(a.f32) - 1) / mark_of(a.f32)) * a.D; }

// The workspace of a call: the backward's partial sums, and the marks where no stash is given.
size_t workspace(Call* c, bool stashed, void* ws) {
  Carver cv(ws);
  c->part = cv.take<float>((size_t)axes(c->a) * kMostShare * c->a.D);
  if (!stashed) c->marks = cv.take<float>((size_t)mark_count(c->a));
  return cv.off;
}

ssd_status check_inputs(const Call& c) {
  const uintptr_t elem = c.a.f32 ? 4 : 2;
  if (!c.x || !c.r || !c.i || !c.lam || (c.a.packed != (c.cu != nullptr))) return SSD_ERR_INVALID_ARG;
  if (!(c.a.scale >= 0.f) || c.a.scale > 3e38f) return SSD_ERR_INVALID_ARG;
  if (off(c.x, elem) || off(c.r, elem) || off(c.i, elem) || off(c.lam, 4) || off(c.h0, 4) || off(c.cu, 4))
    return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}

}  // namespace

ssd_status make_args(const ssd_glr_problem* p, Args* a) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if ((p->io_dtype != SSD_F32 && p->io_dtype != SSD_BF16) || (p->packed != 0 && p->packed != 1)) return SSD_ERR_INVALID_ARG;
  if (p->batch < 1 || p->seqlen < 1 || p->dim < 1 || p->x_stride < 0 || p->r_stride < 0 || p->i_stride < 0)
    return SSD_ERR_INVALID_ARG;
  if (p->seqlen > kMostSteps || p->batch >= kLast || p->dim > kMostStride) return SSD_ERR_SHAPE;
  if (!p->packed && (p->batch > 65535 || p->batch * p->seqlen > 0x7fffffffll)) return SSD_ERR_SHAPE;
  for (const int64_t s : {p->x_stride, p->r_stride, p->i_stride})
    if ((s && s < p->dim) || s > kMostStride) return SSD_ERR_SHAPE;
  *a = Args{};
  a->N = (int)p->batch;
  a->T = (int)p->seqlen;
  a->D = (int)p->dim;
  a->packed = p->packed == 1;
  a->f32 = p->io_dtype == SSD_F32;
  a->xs = p->x_stride ? p->x_stride : p->dim;
  a->rs = p->r_stride ? p->r_stride : p->dim;
  a->is = p->i_stride ? p->i_stride : p->dim;
  return SSD_OK;
}

}  // namespace glr
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_glr_stash_size(const ssd_glr_problem* prob, size_t* bytes) {
  glr::Args a;
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = glr::make_args(prob, &a);
  if (s != SSD_OK) return s;
  *bytes = (size_t)glr::mark_count(a) * 4;
  return SSD_OK;
}

ssd_status ssd_glr_workspace_size(const ssd_glr_problem* prob, int stashed, size_t* bytes) {
  glr::Call c = {};
  if (!bytes) return SSD_ERR_INVALID_ARG;
  const ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  *bytes = glr::workspace(&c, stashed != 0, nullptr);
  return SSD_OK;
}

ssd_status ssd_glr_forward(const ssd_glr_problem* prob, const void* x, const void* r, const void* i, const float* lam,
                           const float* h0, const int32_t* cu_seqlens, float scale, void* y, float* h_final, void* stash,
                           size_t stash_bytes, void* cuda_stream) {
  glr::Call c = {};
  ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.a.scale = scale;
  c.x = x, c.r = r, c.i = i, c.lam = lam, c.h0 = h0, c.cu = cu_seqlens;
  if ((s = glr::check_inputs(c)) != SSD_OK) return s;
  if (!y) return SSD_ERR_INVALID_ARG;
  if (off(y, 16) || off(h_final, 4) || off(stash, 16)) return SSD_ERR_ALIGNMENT;
  if (stash && stash_bytes < (size_t)glr::mark_count(c.a) * 4) return SSD_ERR_WORKSPACE;
  c.y = y, c.h_final = h_final, c.marks = static_cast<float*>(stash);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = glr::forward(c, st);
  return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_glr_backward(const ssd_glr_problem* prob, const void* dy, const float* dh_final, const void* x, const void* r,
                            const void* i, const float* lam, const float* h0, const int32_t* cu_seqlens, float scale,
                            void* dx, void* dr, void* di, float* dlam, float* dh0, const void* stash, size_t stash_bytes,
                            void* ws, size_t ws_bytes, void* cuda_stream) {
  glr::Call c = {};
  ssd_status s = glr::make_args(prob, &c.a);
  if (s != SSD_OK) return s;
  c.a.scale = scale;
  c.x = x, c.r = r, c.i = i, c.lam = lam, c.h0 = h0, c.cu = cu_seqlens;
  if ((s = glr::check_inputs(c)) != SSD_OK) return s;
  if (!dy || !dx || !dr || !di || !dlam || !ws) return SSD_ERR_INVALID_ARG;
  if (off(dy, c.a.f32 ? 4 : 2) || off(dh_final, 4) || off(dx, 16) || off(dr, 16) || off(di, 16) ||
      off(dlam, 4) || off(dh0, 4) || off(stash, 16) || off(ws, 16))
    return SSD_ERR_ALIGNMENT;
  if (stash && stash_bytes < (size_t)glr::mark_count(c.a) * 4) return SSD_ERR_WORKSPACE;
  if (ws_bytes < glr::workspace(&c, stash != nullptr, nullptr)) return SSD_ERR_WORKSPACE;
  glr::workspace(&c, stash != nullptr, ws);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (stash)
    c.marks = const_cast<float*>(static_cast<const float*>(stash));
  else
    e = glr::forward(c, st);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  c.dy = dy, c.dh_final = dh_final, c.dx = dx, c.dr = dr, c.di = di, c.dh0 = dh0;
  int rows = 0;
  e = glr::backward(c, st, &rows);
  if (e != cudaSuccess) return SSD_ERR_CUDA;
  SSD_LAUNCH("k_glr_lam", st,
             glr::k_glr_lam<<<(c.a.D + 31) / 32, dim3(32, rows > 256 ? 32 : 8), 0, st>>>(c.part, rows, c.a.D, lam, dlam));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
