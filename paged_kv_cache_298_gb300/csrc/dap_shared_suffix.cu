// dap_shared_suffix.cu -- the suffix kernel of the shared-prefix decode for TMA-fed tiles (page
// sizes that are multiples of 8).  Kernel: dap_shared.cuh.
#include "dap_shared.cuh"

namespace dap {

dap_status launch_shared_suffix(const SharedArgs &a, cudaStream_t stream, bool *merged) {
    if (a.page_size % 8 != 0) return launch_shared_suffix_gather(a, stream, merged);
    return suffix_dims<false>(a, stream, merged);
}

bool read_errors_shared_suffix(unsigned int *flags, bool clear) { return read_tu_errors(flags, clear); }

}  // namespace dap
