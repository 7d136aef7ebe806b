// The layer norm's kernels on bf16 tensors.
#include "norm_kernels.cuh"

namespace ssd {
namespace norm {
void run_bf16(const Call& c, cudaStream_t st) { by_type<bf16>(c, st); }
}  // namespace norm
}  // namespace ssd
