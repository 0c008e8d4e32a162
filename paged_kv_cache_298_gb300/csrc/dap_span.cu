// dap_span.cu -- attention over spans of the paged cache (sliding windows with sinks, trees of drafted tokens): the
// tile-size rule and the TMA-fed configurations of the warp-level kernel.  Kernels: dap_span.cuh.
#include "dap_span.cuh"

namespace dap {

// 8 / G tokens while they hold the longest run of new tokens, else 16 / G.
int span_tokens_per_tile(int G, int D, int max_q_len) {
    (void)D;
    if (G < 1 || G > 8) return 0;
    return max_q_len <= 8 / G ? 8 / G : 16 / G;
}

dap_status launch_span(const SpanArgs &a, cudaStream_t stream) {
    return a.d.page_size % 8 != 0 ? launch_span_gather(a, stream) : span_dims<false>(a, stream);
}

bool read_errors_span(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
