// The backward pass of the attention over whole sequences, bf16.
#include "attention_bwd.cuh"

namespace gbn {

cudaError_t launch_attention_bwd_bf16(const AttnBwdParams& p, cudaStream_t stream) {
  return launch_bwd<__nv_bfloat16>(p, stream);
}
cudaError_t read_attention_bwd_bf16_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

}  // namespace gbn
