// attn_prefill.hip -- attention of prompts and chunks of prompts over the paged cache.
#include "attn_simple.h"

namespace w4 {

size_t attn_prefill_work_bytes(int64_t, int, const KvView &, int, int) { return 0; }

hipError_t launch_attn_prefill(const AttnArgs &a, const KvView &cache, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(a.n_heads));
    hipLaunchKernelGGL(attn_simple_kernel, grid, dim3(64), 0, stream, a, cache);
    return hipGetLastError();
}

}  // namespace w4
