// dap_span.cu -- attention over spans of the paged cache (sliding windows with sinks, trees of drafted tokens): the
// tile-size rule and the TMA-fed configurations of the warp-level kernel.  Kernels: dap_span.cuh.
#include "dap_span.cuh"

namespace dap {

// 8 / G tokens, or 16 / G, while they hold the longest run of new tokens; beyond that the rows of tensor-memory products
// where the head dim has them.
int span_tokens_per_tile(int G, int D, int max_q_len) {
    if (G < 1 || G > 8) return 0;
    if (max_q_len <= 8 / G) return 8 / G;
    if (max_q_len > 16 / G && (D == 64 || D == 128 || D == 256)) return (D == 256 ? 128 : 256) / G;
    return 16 / G;
}

dap_status launch_span(const SpanArgs &a, cudaStream_t stream) {
    if (a.d.tokens_per_tile * (a.d.Hq / a.d.Hkv) >= 128) return launch_span_tc(a, stream);
    return a.d.page_size % 8 != 0 ? launch_span_gather(a, stream) : span_dims<false>(a, stream);
}

bool read_errors_span(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
