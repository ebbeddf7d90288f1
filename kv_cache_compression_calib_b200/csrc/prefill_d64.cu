// Prompt attention at head dim 64 (kernels and reasons in prefill.cuh; a file per head
// dim so that they compile side by side).
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_d64(const PrefillParams &p, cudaStream_t s) { return launch_d<64>(p, s); }

}  // namespace tri
