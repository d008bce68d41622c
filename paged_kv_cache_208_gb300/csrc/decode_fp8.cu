// decode_fp8.cu -- paged decode attention over the 8-bit cache (the kernel is in
// decode_kernel.cuh, the format in fp8_cache.cuh).
#include "decode_kernel.cuh"

namespace pkv {

cudaError_t launch_paged_decode_fp8(const DecodeArgs &a, const DecodePlan &plan,
                                    cudaStream_t stream) {
  return plan.scores_at ? launch_decode<true, true>(a, plan, stream)
                        : launch_decode<true, false>(a, plan, stream);
}

}  // namespace pkv
