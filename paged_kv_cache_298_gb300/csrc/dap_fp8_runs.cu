// dap_fp8_runs.cu -- runs of tokens in the e4m3 GQA cache: quantising them as they are written
// (kv_append_paged_fp8_multi: prompts, prompt chunks, drafted tokens) and reading them back
// as bf16 rows (kv_read_paged_fp8).
//
// The rows of all sequences are packed back to back: row r belongs to the sequence b with
// indptr[b] <= r < indptr[b + 1] and sits at logical position positions[b] + r - indptr[b], which the
// block table translates as everywhere else.
//   write:  a = max_d |x_d|,  s = bf16(a / 448) (1 for an all-zero row),
//           code_d = e4m3(x_d / s), round to nearest even, saturating;
//   read:   y_d = bf16(e4m3(code_d) * s): the product of 4 and 8 significant bits is exact in
//           binary32, so this is one rounding.
// The factor is taken in binary32 and stored as bf16, the format of the cache; the codes are
// divided by the stored factor, so the rounding of the factor costs no accuracy.
#include <cuda_fp8.h>

#include "dap_tile.cuh"

namespace dap {

namespace {

// The place of packed row r: found by a whole warp, which probes 32 boundaries at once (B up to
// 1024 takes two rounds).  Any contents of indptr keep the accesses inside it.
struct Place {
    bool run, ok;  // the row belongs to a run; its position and page are inside
    int page, slot;
};

__device__ __forceinline__ Place find_place(const RunArgs &p, long long r, int lane) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step;
        const bool le = at < hi && (long long)__ldg(p.indptr + at) <= r;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, le));
        hi = (int)min((long long)hi, lo + (long long)(n + 1) * step);
        lo += n * step;
    }
    const long long i = r - __ldg(p.indptr + lo);
    Place w = {i >= 0 && r < __ldg(p.indptr + lo + 1), false, 0, 0};
    if (!w.run) return w;
    const long long pos = (long long)__ldg(p.positions + lo) + i;
    if (pos < 0 || pos >= (long long)p.max_pages * p.page_size) {
        if (lane == 0) flag_error(DAP_DEVERR_SEQLEN);
        return w;
    }
    w.page = __ldg(p.block_table + (long long)lo * p.max_pages + pos / p.page_size);
    w.slot = (int)(pos % p.page_size);
    w.ok = w.page >= 0 && w.page < p.num_pages;
    if (!w.ok && lane == 0) flag_error(DAP_DEVERR_PAGE);
    return w;
}

// One warp per (row, kv head): D / 32 values a lane.
template <int D>
__global__ void __launch_bounds__(256) append_runs_kernel(const RunArgs p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int V = D / 32;
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= (long long)p.T * p.Hkv) return;
    const long long r = unit / p.Hkv;
    const int h = (int)(unit - r * p.Hkv);
    const Place w = find_place(p, r, lane);
    if (!w.ok) return;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const __nv_bfloat16 *src = p.rows[kv] + r * p.st[kv] + h * p.sh[kv] + lane * V;
        float x[V], amax = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = __bfloat162float(src[i]);
            amax = fmaxf(amax, fabsf(x[i]));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const __nv_bfloat16 s = __float2bfloat16_rn(amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f);
        uint8_t *dst = p.codes[kv] + (((long long)w.page * p.page_size + w.slot) * p.Hkv + h) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i)
            dst[i] = __nv_cvt_float_to_fp8(__fdiv_rn(x[i], __bfloat162float(s)), __NV_SATFINITE, __NV_E4M3);
        if (lane == 0) p.scale[kv][((long long)w.page * p.Hkv + h) * p.page_size + w.slot] = s;
    }
}

template <int D>
__global__ void __launch_bounds__(256) read_runs_kernel(const RunArgs p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int V = D / 32;
    const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (unit >= (long long)p.T * p.Hkv) return;
    const long long r = unit / p.Hkv;
    const int h = (int)(unit - r * p.Hkv);
    const Place w = find_place(p, r, lane);
    if (!w.run) return;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        __nv_bfloat16 *dst = p.rows[kv] + r * p.st[kv] + h * p.sh[kv] + lane * V;
        const uint8_t *src = p.codes[kv] + (((long long)w.page * p.page_size + w.slot) * p.Hkv + h) * D + lane * V;
        const float s =
            w.ok ? __bfloat162float(p.scale[kv][((long long)w.page * p.Hkv + h) * p.page_size + w.slot]) : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float c = w.ok ? __half2float(__half(__nv_cvt_fp8_to_halfraw(src[i], __NV_E4M3))) : 0.f;
            dst[i] = __float2bfloat16_rn(c * s);
        }
    }
}

template <int D>
dap_status launch_d(const RunArgs &a, bool write, cudaStream_t stream) {
    const long long units = (long long)a.T * a.Hkv;
    if ((units + 7) / 8 > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    const dim3 grid((unsigned)((units + 7) / 8));
    const cudaError_t e = write ? launch_dependent(append_runs_kernel<D>, grid, dim3(256), stream, a)
                                : launch_dependent(read_runs_kernel<D>, grid, dim3(256), stream, a);
    return e == cudaSuccess ? DAP_OK : DAP_ERR_CUDA;
}

}  // namespace

dap_status launch_fp8_runs(const RunArgs &a, bool write, cudaStream_t stream) {
    switch (a.D) {
        case 64: return launch_d<64>(a, write, stream);
        case 128: return launch_d<128>(a, write, stream);
        case 256: return launch_d<256>(a, write, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

bool read_errors_fp8_runs(unsigned int *flags, bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_errors, sizeof v) != cudaSuccess) return false;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_device_errors, &z, sizeof z) != cudaSuccess) return false;
    }
    *flags |= v;
    return true;
}

}  // namespace dap
