// Prompt attention: dispatch by head dim, and the size of its scratch.
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_d64(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_d256(const PrefillParams &p, cudaStream_t s);

// Scratch of split rows: at most one part per SM.
size_t prefill_scratch_bytes(int64_t L, int64_t S, int64_t H, int64_t G, int D, int64_t T) {
    const int64_t units = most_blocks(S, G, D, T) * L * H;
    if (units == 0 || units > kMostParts / 2) return 0;
    return (size_t)(kMostParts / units * units) * (D == 256 ? kRows : 2 * kRows) * (D + 2) * sizeof(float);
}

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_prefill_d64(p, s);
        case 128: return launch_prefill_d128(p, s);
        case 256: return launch_prefill_d256(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tri
