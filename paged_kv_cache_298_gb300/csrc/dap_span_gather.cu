// dap_span_gather.cu -- attention over spans of a paged cache whose page size is not a multiple of 8: the configurations
// of dap_span.cuh with the row-gather producer.
#include "dap_span.cuh"

namespace dap {

dap_status launch_span_gather(const SpanArgs &a, cudaStream_t stream) { return span_dims<2, true>(a, stream); }

bool read_errors_span_gather(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
