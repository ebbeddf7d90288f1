// Self-test of the waits of prompt attention at head dim 256: its kernels as they are (prefill.cuh), but
// for when a wait gives up - after the short tries the caller gives, while copies, products and other
// warps' waits are under way, as when one of them never completed.  The block then waits for its
// copies and products and ends with TRI_FLAG_STAGE_TIMEOUT.  No fault is involved.
#define TRI_WAIT_TRY mbar_test_now
#define TRI_WAIT_LOOK(it, p) ((it) >= (p).wait_tries || ((it) & 4095u) == 0)
#define TRI_WAIT_OVER(it, p) ((it) >= (p).wait_tries)
#include "prefill.cuh"

namespace tri {

cudaError_t launch_prefill_selftest_d256(const PrefillParams &p, cudaStream_t s) { return launch_d<256>(p, s); }

}  // namespace tri
