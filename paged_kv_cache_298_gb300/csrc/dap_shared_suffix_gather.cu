// dap_shared_suffix_gather.cu -- the suffix kernel of the shared-prefix decode for page sizes that are
// not multiples of 8 (row-gather producer).  Kernel: dap_shared.cuh.
#include "dap_shared.cuh"

namespace dap {

dap_status launch_shared_suffix_gather(const SharedArgs &a, cudaStream_t stream, bool *merged) {
    return suffix_dims<true>(a, stream, merged);
}

bool read_errors_shared_suffix_gather(unsigned int *flags, bool clear) { return read_tu_errors(flags, clear); }

}  // namespace dap
