// dap_span_few.cu -- attention over spans of the paged cache by few CTAs: the configurations of dap_span.cuh with 64-key tiles.
#include "dap_span.cuh"

namespace dap {

dap_status launch_span_few(const SpanArgs &a, cudaStream_t stream) { return span_dims<4, false>(a, stream); }

bool read_errors_span_few(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
