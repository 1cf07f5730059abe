// The kernel of attn_paged_few.cuh where another launch takes part of a call's tokens.
#include "attn_paged_few.cuh"

namespace qsa {

cudaError_t launch_paged_few_mixed(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream) {
  return launch_few<true>(a, kv_type, err, stream);
}

}  // namespace qsa
