// The calls of the layer norm, and the last step of its weight gradient (the kernels: norm_kernels.cuh).
#include <initializer_list>

#include "norm_common.cuh"
#include "ssd.h"

namespace ssd {
namespace norm {
namespace {

// out[c] = sum over n blocks of part[.][c]: 32 columns a block, 32 rows at a time; blockIdx.y: dw, db.
__global__ void __launch_bounds__(1024) k_norm_columns(const float* __restrict__ part, int n, int D, void* dw, void* db,
                                                        bool wbf16) {
  __shared__ float s[32][33];
  void* out = blockIdx.y ? db : dw;
  if (!out) return;
  const float* p = part + (size_t)blockIdx.y * n * D;
  const int c = blockIdx.x * 32 + threadIdx.x;
  float x = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int i = threadIdx.y; i < n; i += 32) x += p[(size_t)i * D + c];
  }
  s[threadIdx.y][threadIdx.x] = x;
  __syncthreads();
  x = s[threadIdx.x][threadIdx.y];  // one column a warp
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < D) {
    if (wbf16)
      static_cast<bf16*>(out)[col] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(out)[col] = x;
  }
}

void run(const Call& c, bool f32, cudaStream_t st) {
  if (f32)
    run_f32(c, st);
  else
    run_bf16(c, st);
  if (c.part)
    SSD_LAUNCH("k_norm_columns", st,
               k_norm_columns<<<dim3((unsigned)((c.a.D + 31) / 32), 2), dim3(32, 32), 0, st>>>(
                   c.part, backward_blocks(c.a.rows, c.a.D, f32), c.a.D, c.dw, c.db, c.a.wbf16));
}

ssd_status make(const ssd_norm_problem* p, Call* c, bool* f32) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if ((p->io_dtype != SSD_F32 && p->io_dtype != SSD_BF16) || (p->weight_dtype != SSD_F32 && p->weight_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  if (p->rows < 1 || p->dim < 1 || p->x_stride < 0) return SSD_ERR_INVALID_ARG;
  if (p->dim > 16384 || p->rows > 0x7fffffffll || (p->x_stride && p->x_stride < p->dim)) return SSD_ERR_SHAPE;
  *c = Call{};
  c->a.rows = p->rows;
  c->a.D = (int)p->dim;
  c->a.xs = p->x_stride ? p->x_stride : p->dim;
  c->a.wbf16 = p->weight_dtype == SSD_BF16;
  *f32 = p->io_dtype == SSD_F32;
  return SSD_OK;
}

ssd_status check(std::initializer_list<const void*> req, std::initializer_list<const void*> opt) {
  for (const void* p : req)
    if (!p) return SSD_ERR_INVALID_ARG;
  for (const void* p : req)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SSD_ERR_ALIGNMENT;
  for (const void* p : opt)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return SSD_ERR_ALIGNMENT;
  return SSD_OK;
}

size_t workspace(const Call& c, bool f32) {
  Carver cv(nullptr);
  cv.take<float>(2 * (size_t)backward_blocks(c.a.rows, c.a.D, f32) * c.a.D);
  return cv.off;
}

}  // namespace
}  // namespace norm
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_norm_workspace_size(const ssd_norm_problem* prob, size_t* bytes) {
  if (!bytes) return SSD_ERR_INVALID_ARG;
  norm::Call c;
  bool f32;
  const ssd_status s = norm::make(prob, &c, &f32);
  if (s != SSD_OK) return s;
  *bytes = norm::workspace(c, f32);
  return SSD_OK;
}

ssd_status ssd_norm_forward(const ssd_norm_problem* prob, const void* x, const void* weight, const void* bias, float eps,
                            void* y, float* mean, float* rstd, void* cuda_stream) {
  norm::Call c;
  bool f32;
  ssd_status s = norm::make(prob, &c, &f32);
  if (s != SSD_OK) return s;
  if ((s = norm::check({y}, {weight, bias})) != SSD_OK) return s;
  if (!x) return SSD_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(x) % (f32 ? 4 : 2) || reinterpret_cast<uintptr_t>(mean) % 4 ||
      reinterpret_cast<uintptr_t>(rstd) % 4)
    return SSD_ERR_ALIGNMENT;
  if (!(eps >= 0.f)) return SSD_ERR_INVALID_ARG;
  c.a.eps = eps;
  c.x = x;
  c.w = weight;
  c.b = bias;
  c.y = y;
  c.mean = mean;
  c.rstd = rstd;
  norm::run(c, f32, static_cast<cudaStream_t>(cuda_stream));
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_norm_backward(const ssd_norm_problem* prob, const void* dy, const void* x, const float* mean,
                             const float* rstd, const void* weight, void* dx, void* dw, void* db, void* ws,
                             size_t ws_bytes, void* cuda_stream) {
  norm::Call c;
  bool f32;
  ssd_status s = norm::make(prob, &c, &f32);
  if (s != SSD_OK) return s;
  if ((s = norm::check({dy, dx}, {weight, dw, db, ws})) != SSD_OK) return s;
  if (!x || !mean || !rstd) return SSD_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(x) % (f32 ? 4 : 2) || reinterpret_cast<uintptr_t>(mean) % 4 ||
      reinterpret_cast<uintptr_t>(rstd) % 4)
    return SSD_ERR_ALIGNMENT;
  if (dw || db) {
    if (!ws) return SSD_ERR_INVALID_ARG;
    if (ws_bytes < norm::workspace(c, f32)) return SSD_ERR_WORKSPACE;
    Carver cv(ws);
    c.part = cv.take<float>(2 * (size_t)norm::backward_blocks(c.a.rows, c.a.D, f32) * c.a.D);
  }
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  c.dy = dy;
  c.x = x;
  c.mean = const_cast<float*>(mean);
  c.rstd = const_cast<float*>(rstd);
  c.w = weight;
  c.dx = dx;
  c.dw = dw;
  c.db = db;
  c.backward = true;
  norm::run(c, f32, st);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
