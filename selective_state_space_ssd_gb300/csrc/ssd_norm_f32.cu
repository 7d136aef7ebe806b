// The layer norm's kernels on fp32 tensors.
#include "norm_kernels.cuh"

namespace ssd {
namespace norm {
void run_f32(const Call& c, cudaStream_t st) { by_type<float>(c, st); }
}  // namespace norm
}  // namespace ssd
