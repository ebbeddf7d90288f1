// Prompt attention at head dim 256 (kernels and reasons in prefill.cuh; a file per head
// dim so that they compile side by side).
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_d256(const PrefillParams &p, cudaStream_t s) { return launch_d<256>(p, s); }

}  // namespace tri
