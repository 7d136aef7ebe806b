// What the files of the layer norm share: a call's arguments and how its rows are laid over threads.
#pragma once

#include <cuda_bf16.h>

#include "ssd_internal.h"

namespace ssd {
namespace norm {

using bf16 = __nv_bfloat16;

struct Args {
  long long rows, xs;  // rows; elements from a row of x to the next
  int D;
  bool wbf16;
  float eps;
};

struct Call {
  Args a;
  const void *dy, *x, *w, *b;
  void *y, *dx, *dw, *db;
  float *mean, *rstd, *part;
  bool backward;
};

// Threads a row and elements a thread: the fewest threads, from 8 to 512, that hold a row with at most 40 elements each
// (24 in fp32, whose next row takes twice the registers), in eights: 2560 bf16 values are 64 threads of 40, a head's 128
// are eight threads of 16.  Fewer threads a row mean fewer steps of the sums across them and fewer idle ones.
struct Shape {
  int tpr, e;
};
inline Shape shape_of(int D, bool f32) {
  const int most = f32 ? 24 : 40;
  int t = 8;
  while (t < 512 && t * most < D) t *= 2;
  return Shape{t, (D + 8 * t - 1) / (8 * t) * 8};
}

// Blocks of the backward, each with a row of partial sums: as many as this GPU's 152 SMs hold at once, four an SM at
// most.
inline int backward_blocks(long long rows, int D, bool f32) {
  const Shape s = shape_of(D, f32);
  const int threads = s.tpr < 128 ? 128 : s.tpr, regs = (f32 ? 6 : 5) * s.e + 48;
  int per = 65536 / (threads * (regs < 255 ? regs : 255));
  per = per < 1 ? 1 : per > 4 ? 4 : per;
  const long long groups = threads / s.tpr, want = (rows + groups - 1) / groups, most = 152 * per;
  return (int)(want < most ? want : most);
}

// The kernels of a call, by the type of x (ssd_norm_bf16.cu, ssd_norm_f32.cu).
void run_bf16(const Call& c, cudaStream_t st);
void run_f32(const Call& c, cudaStream_t st);

}  // namespace norm
}  // namespace ssd
