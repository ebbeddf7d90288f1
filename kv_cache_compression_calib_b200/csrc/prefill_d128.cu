// Prompt attention at head dim 128 (kernels and reasons in prefill.cuh; a file per head
// dim so that they compile side by side).
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_d128(const PrefillParams &p, cudaStream_t s) { return launch_d<128>(p, s); }

}  // namespace tri
