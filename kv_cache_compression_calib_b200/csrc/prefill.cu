// Prompt attention: dispatch by head dim, and the size of its scratch.
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_d64(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_d256(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_selftest_d64(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_selftest_d256(const PrefillParams &p, cudaStream_t s);

namespace {
size_t part_bytes(int D) { return (size_t)(D == 256 ? kRows : 2 * kRows) * (D + 2) * sizeof(float); }
}  // namespace

// Scratch of split rows: at most one part per SM.
size_t prefill_scratch_bytes(int64_t L, int64_t S, int64_t H, int64_t G, int D, int64_t T) {
    if (T == 0 || T > kMostParts * kRows || L * H > kMostParts / 2) return 0;  // (more units than that)
    const int64_t units = most_blocks(S, G, D, T) * L * H;
    return units > kMostParts / 2 ? 0 : kMostParts / units * units * part_bytes(D);
}

// What no call of fewer sequences or tokens exceeds: those are split into more parts.
size_t prefill_scratch_most(int64_t L, int64_t H, int64_t G, int D, int64_t T) {
    if (T == 0 || L * H > kMostParts / 2 || most_blocks(1, G, D, 1) * L * H > kMostParts / 2) return 0;
    return kMostParts * part_bytes(D);
}

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_prefill_d64(p, s);
        case 128: return launch_prefill_d128(p, s);
        case 256: return launch_prefill_d256(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_prefill_selftest(const PrefillParams &p, cudaStream_t s) {
    switch (p.geo.D) {
        case 64: return launch_prefill_selftest_d64(p, s);
        case 256: return launch_prefill_selftest_d256(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tri
