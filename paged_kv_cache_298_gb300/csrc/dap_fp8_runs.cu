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
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dap_tile.cuh"

namespace dap {

namespace {

// Both kernels are bound by memory (3 D + 2 bytes a row).  A CTA takes TT consecutive tokens x all kv heads of K
// and V, so that a place is looked up once for 2 Hkv rows, a token's codes (Hkv D bytes) are read or written in
// one place and the factors of neighbouring slots meet in one store.  CTAs of four warps, so that the registers of
// the loads ahead fit seven to an SM and the last ones fill it evenly.  Measured: 50,000 tokens of 8 kv heads x 128
// written in 49.6 us (309 MB, 0.92 of the copy rate; with 256 threads, four CTAs to an SM and the addresses multiplied
// out a row: 55 us), 40,000 read back in 40 us (249 MB, 0.91), 7700 written in 10.9 us and 8000 of 4 heads x 256 read in
// 8.3, of which 3 are the launch.
constexpr int kMaxTT = 64, kThreads = 128;

// Sequence of packed row r, found by a whole warp that probes 32 boundaries at once (B up to 1024
// takes two rounds); any contents of indptr keep the accesses inside it.
__device__ __forceinline__ int find_run(const int32_t *indptr, int B, int r, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && indptr[at] <= r));
        hi = (int)min((long long)hi, lo + (long long)(n + 1) * step);
        lo += n * step;
    }
    return lo;
}

// Where tokens r0 .. r0 + n - 1 are, one per thread of the first warps: element of their first code (-1 where the row
// is in no run, -2 where its position or page is outside, which is flagged) and of kv head 0's factor.
struct Places {
    long long code[kMaxTT], factor[kMaxTT];
};
__device__ __forceinline__ void find_places(const RunArgs &p, int r0, int n, Places &place) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = warp * 32;
    if (first >= n) return;
    const int cnt = min(32, n - first);
    // the run of the warp's first and last token; usually one, else each lane searches between the two
    int lo = find_run(p.indptr, p.B, r0 + first, lane);
    int hi = cnt > 1 && p.B > 1 ? find_run(p.indptr, p.B, r0 + first + cnt - 1, lane) : lo;
    if (lane >= cnt) return;
    const int r = r0 + first + lane;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.indptr[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    const long long b0 = p.indptr[lo], b1 = p.indptr[lo + 1], start = p.positions[lo];
    long long code = -1, factor = 0;
    if (r >= b0 && r < b1) {
        const long long pos = start + (r - b0);
        code = -2;
        if (pos >= 0 && pos < (long long)p.max_pages * p.page_size) {
            // (a position below 2^32, as a run starts at an int32 and has fewer than 2^31 rows)
            const int pg = (int)((uint32_t)pos / (uint32_t)p.page_size);
            const int slot = (int)((uint32_t)pos - (uint32_t)pg * (uint32_t)p.page_size);
            const int page = p.block_table[(long long)lo * p.max_pages + pg];
            if (page >= 0 && page < p.num_pages) {
                code = ((long long)page * p.page_size + slot) * (p.Hkv * p.D);
                factor = (long long)page * p.Hkv * p.page_size + slot;
            } else {
                flag_error(DAP_DEVERR_PAGE);
            }
        } else {
            flag_error(DAP_DEVERR_SEQLEN);
        }
    }
    place.code[first + lane] = code;
    place.factor[first + lane] = factor;
}

// Token and head of the rows that a lane takes, RPP apart: one division, then steps of (RPP / Hkv, RPP % Hkv).
struct RowStep {
    int tok, head, dq, dr, Hkv;
    __device__ __forceinline__ RowStep(int i, int step, int Hkv_) : Hkv(Hkv_) {
        tok = i / Hkv;
        head = i - tok * Hkv;
        dq = step / Hkv;
        dr = step - dq * Hkv;
    }
    __device__ __forceinline__ void next() {
        tok += dq;
        head += dr;
        if (head >= Hkv) {
            head -= Hkv;
            ++tok;
        }
    }
};

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ __nv_bfloat162 habs2(uint32_t w) {
    w &= 0x7FFF7FFFu;
    return *reinterpret_cast<const __nv_bfloat162 *>(&w);
}

// Four values -> four codes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}

// 8 values divided by s by the hardware's rules (by value: the common path keeps its codes in registers).
__device__ __noinline__ uint2 slow_codes(uint4 w, float s) {
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y), c = bf16x2_to_float2(w.z),
                 d = bf16x2_to_float2(w.w);
    return make_uint2(e4m3x4(make_float2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s)),
                             make_float2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s))),
                      e4m3x4(make_float2(__fdiv_rn(c.x, s), __fdiv_rn(c.y, s)),
                             make_float2(__fdiv_rn(d.x, s), __fdiv_rn(d.y, s))));
}

// Write: D / 16 lanes a row, two chunks of 8 values (16 bytes) each; a lane takes the K row and the V row of
// one (token, head), which share their place, and loads the next pair before it works on this one.  The first
// rows are loaded before any place is looked up (their address does not depend on it).  The maximum is taken
// on bf16 pairs, which is exact and skips NaN as fmaxf does.
// A quotient x / y is one product with the approximate reciprocal and one correction step (q -= (q y - x) / y,
// the remainder exact in a fused multiply-add): within 2^-44 of itself before its last rounding.  Code: a
// quotient that binary32 holds (every tie between two codes is one) comes out exactly, and any other lies at
// least 2^-14 of itself from a tie.  Factor: 8 bits over 7, which binary32 holds or which lies at least 2^-28
// from where its rounding changes.  Rows with a maximum outside [2^-90, 2^90], where the steps could leave the
// normal range, are divided by the hardware's rules.
template <int D>
__global__ void __launch_bounds__(kThreads, 7) append_runs_kernel(const RunArgs p, const int TT) {
    constexpr int LPR = D / 16, RPP = kThreads / LPR;
    __shared__ Places place;
    extern __shared__ __nv_bfloat16 factor[];  // [2][Hkv][TT]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int r0 = blockIdx.x * TT, n = min(TT, p.T - r0);
    const int c = threadIdx.x % LPR;
    RowStep at(threadIdx.x / LPR, RPP, p.Hkv);
    const __nv_bfloat16 *k = p.rows[0] + c * 8 + (r0 + (long long)at.tok) * p.st[0] + at.head * p.sh[0];
    const __nv_bfloat16 *v = p.rows[1] + c * 8 + (r0 + (long long)at.tok) * p.st[1] + at.head * p.sh[1];
    // (their steps with `at`: within the heads, and over to the next token)
    const long long ka = at.dq * p.st[0] + at.dr * p.sh[0], kb = ka + p.st[0] - p.Hkv * p.sh[0];
    const long long va = at.dq * p.st[1] + at.dr * p.sh[1], vb = va + p.st[1] - p.Hkv * p.sh[1];
    uint4 next[4];
    auto load = [&] {  // the K row and the V row at (at.tok, at.head)
        if (at.tok < n) {
            next[0] = *reinterpret_cast<const uint4 *>(k);
            next[1] = *reinterpret_cast<const uint4 *>(k + D / 2);
            next[2] = *reinterpret_cast<const uint4 *>(v);
            next[3] = *reinterpret_cast<const uint4 *>(v + D / 2);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) next[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load();
    find_places(p, r0, n, place);
    __syncthreads();
    while (__any_sync(0xFFFFFFFFu, at.tok < n)) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = next[u];
        const int tok = at.tok, head = at.head;
        const bool wrap = at.head + at.dr >= p.Hkv;
        k += wrap ? kb : ka;
        v += wrap ? vb : va;
        at.next();
        load();
        const bool live = tok < n;
        const long long code0 = live ? place.code[tok] : -1, off = code0 + (head * D + c * 8);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t w[8] = {x[2 * kv].x,     x[2 * kv].y,     x[2 * kv].z,     x[2 * kv].w,
                                   x[2 * kv + 1].x, x[2 * kv + 1].y, x[2 * kv + 1].z, x[2 * kv + 1].w};
            __nv_bfloat162 m2 = habs2(w[0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) m2 = __hmax2(m2, habs2(w[k]));
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) m2 = __hmax2(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
            const float amax = fmaxf(__bfloat162float(m2.x), __bfloat162float(m2.y));
            uint32_t code[4];
            __nv_bfloat16 s16;
            if (amax >= 0x1p-90f && amax <= 0x1p90f) {
                constexpr float c448 = 1.f / 448.f;
                const float q0 = amax * c448;
                s16 = __float2bfloat16_rn(fmaf(fmaf(q0, 448.f, -amax), -c448, q0));
                const float s = __bfloat162float(s16), rc = rcp(s);
                const float2 r2 = make_float2(rc, rc), n2 = make_float2(-rc, -rc), s2 = make_float2(s, s);
                const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {  // (this order of signs keeps the sign of a zero)
                    const float2 a = bf16x2_to_float2(w[k]), b = bf16x2_to_float2(w[k + 1]);
                    const float2 qa = __fmul2_rn(a, r2), qb = __fmul2_rn(b, r2);
                    code[k / 2] = e4m3x4(__ffma2_rn(__ffma2_rn(qa, s2, __fmul2_rn(a, minus)), n2, qa),
                                         __ffma2_rn(__ffma2_rn(qb, s2, __fmul2_rn(b, minus)), n2, qb));
                }
            } else {
                s16 = __float2bfloat16_rn(amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f);
                const uint2 a = slow_codes(x[2 * kv], __bfloat162float(s16));
                const uint2 b = slow_codes(x[2 * kv + 1], __bfloat162float(s16));
                code[0] = a.x;
                code[1] = a.y;
                code[2] = b.x;
                code[3] = b.y;
            }
            if (code0 >= 0) {
                uint8_t *dst = p.codes[kv] + off;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
                *reinterpret_cast<uint2 *>(dst + D / 2) = make_uint2(code[2], code[3]);
            }
            if (live && c == 0) factor[(kv * p.Hkv + head) * TT + tok] = s16;
        }
    }
    __syncthreads();
    // the factors head by head: neighbouring threads write neighbouring slots
    for (int i = threadIdx.x; i < n * p.Hkv; i += kThreads) {
        const int h = i / n, t = i - h * n;
        if (place.code[t] >= 0) {
            const long long at_page = place.factor[t] + (long long)h * p.page_size;
            p.scale[0][at_page] = factor[h * TT + t];
            p.scale[1][at_page] = factor[(p.Hkv + h) * TT + t];
        }
    }
}

// Read: D / 16 lanes a row, two chunks of 8 codes (8 bytes read, 16 written) each, so that a warp's stores are
// whole sectors; a lane takes the K row and the V row of one (token, head), U pairs in flight.
template <int D>
__global__ void __launch_bounds__(kThreads, 10) read_runs_kernel(const RunArgs p, const int TT) {
    constexpr int LPR = D / 16, RPP = kThreads / LPR, U = 2;
    __shared__ Places place;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int r0 = blockIdx.x * TT, n = min(TT, p.T - r0);
    const int c = threadIdx.x % LPR;
    RowStep at(threadIdx.x / LPR, RPP, p.Hkv);
    find_places(p, r0, n, place);
    __syncthreads();
    while (at.tok < n) {
        uint2 x[U][2][2];
        float s[U][2];
        int tok[U], head[U];
        bool run[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tok[u] = at.tok;
            head[u] = at.head;
            at.next();
            const long long code0 = tok[u] < n ? place.code[tok[u]] : -1;
            run[u] = code0 != -1;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                x[u][kv][0] = x[u][kv][1] = make_uint2(0u, 0u);
                s[u][kv] = 0.f;
            }
            if (code0 >= 0) {
                const long long off = code0 + (head[u] * D + c * 8);
                const long long f = place.factor[tok[u]] + (long long)head[u] * p.page_size;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    x[u][kv][0] = *reinterpret_cast<const uint2 *>(p.codes[kv] + off);
                    x[u][kv][1] = *reinterpret_cast<const uint2 *>(p.codes[kv] + off + D / 2);
                    s[u][kv] = __bfloat162float(p.scale[kv][f]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!run[u]) continue;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const float2 s2 = make_float2(s[u][kv], s[u][kv]);
                __nv_bfloat16 *dst =
                    p.rows[kv] + (long long)(r0 + tok[u]) * p.st[kv] + head[u] * p.sh[kv] + c * 8;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t w[2] = {x[u][kv][hf].x, x[u][kv][hf].y};
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2_raw h =
                            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
                        const float2 f = __fmul2_rn(__half22float2(__half2(h)), s2);
                        y[k] = pack_bf16x2(f.x, f.y);
                    }
                    *reinterpret_cast<uint4 *>(dst + hf * (D / 2)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
}

template <int D>
dap_status launch_d(const RunArgs &a, bool write, cudaStream_t stream) {
    // Tokens of a CTA: a read, two passes of its lanes over the rows (all in flight at once); a write, whose loads
    // run one pass ahead, one pass or up to eight while the grid stays above one wave of seven CTAs per SM
    constexpr int RPP = kThreads * 16 / D;
    if (write && a.Hkv > 10240) return DAP_ERR_UNSUPPORTED;  // (the factors of one token take over 40 KB)
    int passes = 2;
    if (write) {
        const int sms = dap_device_sm_count();
        if (sms <= 0) return DAP_ERR_CUDA;
        const long long rows = (long long)a.T * a.Hkv, wave = (long long)RPP * 7 * sms;
        passes = (int)std::min<long long>(8, std::max<long long>(1, (rows + wave - 1) / wave));
    }
    const int TT = std::min(kMaxTT, std::max(1, passes * RPP / a.Hkv));
    const dim3 grid((unsigned)((a.T + (long long)TT - 1) / TT));
    const size_t smem = write ? (size_t)2 * a.Hkv * TT * sizeof(__nv_bfloat16) : 0;
    const cudaError_t e =
        write ? launch_dependent_smem(append_runs_kernel<D>, grid, dim3(kThreads), (int)smem, stream, a, TT)
              : launch_dependent_smem(read_runs_kernel<D>, grid, dim3(kThreads), (int)smem, stream, a, TT);
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
