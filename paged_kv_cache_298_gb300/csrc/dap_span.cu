// dap_span.cu -- attention over spans of the paged cache (sliding windows with sinks, trees of drafted tokens): the
// tile-size rule and the TMA-fed configurations of the warp-level kernel.  Kernels: dap_span.cuh.
#include "dap_span.cuh"

namespace dap {

// 8 / G tokens, or 16 / G, while they hold the longest run of new tokens; beyond that the rows of tensor-memory products
// where the head dim has them: 128, of which two CTAs share an SM and cover each other's start and end (four chunks of 1021
// tokens behind a window of 2048: 144 us, in tiles of 256 rows 156), or 256 where they and not 128 hold the run, which reads
// its K/V once, from twice as many (sequence, kv head) units as SMs on (64 trees of 64 nodes, G = 4, behind 256 .. 4096 keys:
// 151 us, in tiles of 128 rows 171; 3 of them behind 300 keys 16.3 and 14.3).
int span_tokens_per_tile(int sms, int B, int Hkv, int G, int D, int max_q_len) {
    if (G < 1 || G > 8) return 0;
    if (max_q_len <= 8 / G) return 8 / G;
    if (max_q_len <= 16 / G || !(D == 64 || D == 128 || D == 256)) return 16 / G;
    const bool wide = D < 256 && max_q_len > 128 / G && max_q_len <= 256 / G && (long long)B * Hkv >= 2LL * sms;
    return (wide ? 256 : 128) / G;
}

// 64-key tiles where their CTAs, two an SM (one at D = 256), all run at once.
bool span_few(int sms, long long ctas, int D) { return ctas <= (D == 256 ? 1LL : 2LL) * sms; }

dap_status launch_span(const SpanArgs &a, cudaStream_t stream) {
    if (a.d.tokens_per_tile * (a.d.Hq / a.d.Hkv) >= 128) return launch_span_tc(a, stream);
    const bool gather = a.d.page_size % 8 != 0;
    if (span_few(dap_device_sm_count(), (long long)a.d.num_tiles * a.d.Hkv * a.d.num_splits, a.d.D))
        return gather ? launch_span_few_gather(a, stream) : launch_span_few(a, stream);
    return gather ? launch_span_gather(a, stream) : span_dims<2, false>(a, stream);
}

bool read_errors_span(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
