// The kernel of attn_paged_few.cuh for all tokens of a call.
#include "attn_paged_few.cuh"

namespace qsa {

cudaError_t launch_paged_few(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream) {
  return launch_few<false>(a, kv_type, err, stream);
}

}  // namespace qsa
