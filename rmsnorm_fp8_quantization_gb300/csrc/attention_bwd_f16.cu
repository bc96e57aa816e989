// The backward pass of the attention over whole sequences, f16.
#include "attention_bwd.cuh"

namespace gbn {

cudaError_t launch_attention_bwd_f16(const AttnBwdParams& p, cudaStream_t stream) {
  return launch_bwd<__half>(p, stream);
}
cudaError_t read_attention_bwd_f16_error(unsigned int* v, bool clear) { return read_paged_error(v, clear); }

}  // namespace gbn
