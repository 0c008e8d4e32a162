// dap_span_few_gather.cu -- attention over spans of the paged cache by few CTAs and page sizes that are not multiples of 8: the configurations of dap_span.cuh
// with 64-key tiles and the row-gather producer.
#include "dap_span.cuh"

namespace dap {

dap_status launch_span_few_gather(const SpanArgs &a, cudaStream_t stream) { return span_dims<4, true>(a, stream); }

bool read_errors_span_few_gather(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
