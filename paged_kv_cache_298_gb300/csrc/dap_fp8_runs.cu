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

// Both kernels are bound by memory (3 D + 2 bytes a row).  A CTA takes TT consecutive tokens x all kv
// heads of K or of V (blockIdx.y), about BATCH rows, so that a token's codes (Hkv D bytes) are read or
// written in one place and the factors of neighbouring slots meet in one store; all loads of a batch
// are in flight before the first is used.
constexpr int kMaxTT = 64;

// Sequence of packed row r, found by a whole warp that probes 32 boundaries at once (B up to 1024
// takes two rounds); any contents of indptr keep the accesses inside it.
__device__ __forceinline__ int find_run(const int32_t *indptr, int B, int r, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const long long at = lo + (long long)(lane + 1) * step;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && __ldg(indptr + at) <= r));
        hi = (int)min((long long)hi, lo + (long long)(n + 1) * step);
        lo += n * step;
    }
    return lo;
}

// Slot of the pool (page * page_size + slot in the page) of tokens r0 .. r0 + n - 1, one per thread of the
// first warps: -1 where the row is in no run, -2 where its position or page is outside (flagged once, by the
// CTAs of K); and the slot in its page.
struct Places {
    long long row[kMaxTT];
    int slot[kMaxTT];
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
        if (__ldg(p.indptr + mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    const long long b0 = __ldg(p.indptr + lo), b1 = __ldg(p.indptr + lo + 1), start = __ldg(p.positions + lo);
    long long row = -1;
    int slot = 0;
    if (r >= b0 && r < b1) {
        const long long pos = start + (r - b0);
        row = -2;
        if (pos >= 0 && pos < (long long)p.max_pages * p.page_size) {
            // (a position below 2^32, as a run starts at an int32 and has fewer than 2^31 rows)
            const int pg = (int)((uint32_t)pos / (uint32_t)p.page_size);
            slot = (int)((uint32_t)pos - (uint32_t)pg * (uint32_t)p.page_size);
            const int page = __ldg(p.block_table + (long long)lo * p.max_pages + pg);
            if (page >= 0 && page < p.num_pages) row = (long long)page * p.page_size + slot;
            else if (blockIdx.y == 0) flag_error(DAP_DEVERR_PAGE);
        } else if (blockIdx.y == 0) {
            flag_error(DAP_DEVERR_SEQLEN);
        }
    }
    place.row[first + lane] = row;
    place.slot[first + lane] = slot;
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

// Write: D / 8 lanes a row, 8 values (16 bytes) each, U rows a lane in flight.  The rows are loaded before
// their places are looked up (their address does not depend on them).
// A quotient x / y is one product with the approximate reciprocal and one correction step (q -= (q y - x) / y,
// the remainder exact in a fused multiply-add): within 2^-44 of itself before its last rounding.  Code: a
// quotient that binary32 holds (every tie between two codes is one) comes out exactly, and any other lies at
// least 2^-14 of itself from a tie.  Factor: 8 bits over 7, which binary32 holds or which lies at least 2^-28
// from where its rounding changes.  Rows with a maximum outside [2^-90, 2^90], where the steps could leave the
// normal range, are divided by the hardware's rules.
template <int D>
__global__ void __launch_bounds__(256) append_runs_kernel(const RunArgs p, const int TT) {
    constexpr int LPR = D / 8, RPP = 256 / LPR, U = 4;
    __shared__ Places place;
    extern __shared__ __nv_bfloat16 factor[];  // [Hkv][TT]
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int kv = blockIdx.y;
    const int r0 = blockIdx.x * TT, n = min(TT, p.T - r0), rows = n * p.Hkv;
    const int sub = threadIdx.x / LPR, c = threadIdx.x % LPR;
    const long long st = kv ? p.st[1] : p.st[0], sh = kv ? p.sh[1] : p.sh[0];
    const __nv_bfloat16 *src = (kv ? p.rows[1] : p.rows[0]) + c * 8 + (long long)r0 * st;
    uint8_t *codes = (kv ? p.codes[1] : p.codes[0]) + c * 8;
    RowStep at(sub, RPP, p.Hkv);
    for (int base = 0; base < rows; base += RPP * U) {
        uint4 x[U];
        int tok[U], head[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tok[u] = at.tok;
            head[u] = at.head;
            at.next();
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (tok[u] < n) x[u] = *reinterpret_cast<const uint4 *>(src + tok[u] * st + head[u] * sh);
        }
        if (base == 0) {
            find_places(p, r0, n, place);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            float2 f[4];
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[k] = bf16x2_to_float2(w[k]);
                amax = fmaxf(amax, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
            }
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            __nv_bfloat16 s16;
            if (amax >= 0x1p-90f && amax <= 0x1p90f) {
                constexpr float c448 = 1.f / 448.f;
                const float q0 = amax * c448;
                s16 = __float2bfloat16_rn(fmaf(fmaf(q0, 448.f, -amax), -c448, q0));
                const float s = __bfloat162float(s16), rc = rcp(s);
                const float2 r2 = make_float2(rc, rc), n2 = make_float2(-rc, -rc), s2 = make_float2(s, s);
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // (this order of signs keeps the sign of a zero)
                    const float2 q = __fmul2_rn(f[k], r2);
                    f[k] = __ffma2_rn(__ffma2_rn(q, s2, make_float2(-f[k].x, -f[k].y)), n2, q);
                }
            } else {
                s16 = __float2bfloat16_rn(amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f);
                const float s = __bfloat162float(s16);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = make_float2(__fdiv_rn(f[k].x, s), __fdiv_rn(f[k].y, s));
            }
            uint32_t code[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                code[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(f[2 * k], __NV_SATFINITE, __NV_E4M3) |
                          (uint32_t)__nv_cvt_float2_to_fp8x2(f[2 * k + 1], __NV_SATFINITE, __NV_E4M3) << 16;
            if (tok[u] < n) {
                const long long row = place.row[tok[u]];
                if (row >= 0)
                    *reinterpret_cast<uint2 *>(codes + (row * p.Hkv + head[u]) * D) = make_uint2(code[0], code[1]);
                if (c == 0) factor[head[u] * TT + tok[u]] = s16;
            }
        }
    }
    __syncthreads();
    // the factors head by head: neighbouring threads write neighbouring slots
    __nv_bfloat16 *scale = kv ? p.scale[1] : p.scale[0];
    for (int i = threadIdx.x; i < rows; i += 256) {
        const int h = i / n, t = i - h * n;
        const long long row = place.row[t];
        const int slot = place.slot[t];
        if (row >= 0) scale[(row - slot) * p.Hkv + (long long)h * p.page_size + slot] = factor[h * TT + t];
    }
}

// Read: D / 16 lanes a row, 16 codes (16 bytes) each.
template <int D>
__global__ void __launch_bounds__(256) read_runs_kernel(const RunArgs p, const int TT) {
    constexpr int LPR = D / 16, RPP = 256 / LPR, U = 4;
    __shared__ Places place;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int kv = blockIdx.y;
    const int r0 = blockIdx.x * TT, n = min(TT, p.T - r0), rows = n * p.Hkv;
    const int sub = threadIdx.x / LPR, c = threadIdx.x % LPR;
    const long long st = kv ? p.st[1] : p.st[0], sh = kv ? p.sh[1] : p.sh[0];
    __nv_bfloat16 *out = (kv ? p.rows[1] : p.rows[0]) + c * 16 + (long long)r0 * st;
    const uint8_t *codes = (kv ? p.codes[1] : p.codes[0]) + c * 16;
    const __nv_bfloat16 *scale = kv ? p.scale[1] : p.scale[0];
    RowStep at(sub, RPP, p.Hkv);
    find_places(p, r0, n, place);
    __syncthreads();
    for (int base = 0; base < rows; base += RPP * U) {
        uint4 x[U];
        float s[U];
        int tok[U], head[U];
        bool run[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tok[u] = at.tok;
            head[u] = at.head;
            at.next();
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            s[u] = 0.f;
            run[u] = false;
            if (tok[u] < n) {
                const long long row = place.row[tok[u]];
                run[u] = row != -1;
                if (row >= 0) {
                    const int slot = place.slot[tok[u]];
                    x[u] = *reinterpret_cast<const uint4 *>(codes + (row * p.Hkv + head[u]) * D);
                    s[u] = __bfloat162float(scale[(row - slot) * p.Hkv + (long long)head[u] * p.page_size + slot]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t y[8];
            const float2 s2 = make_float2(s[u], s[u]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const __half2_raw h =
                        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k] >> (16 * hf)), __NV_E4M3);
                    const float2 f = __fmul2_rn(__half22float2(__half2(h)), s2);
                    y[2 * k + hf] = pack_bf16x2(f.x, f.y);
                }
            }
            if (run[u]) {
                uint4 *dst = reinterpret_cast<uint4 *>(out + tok[u] * st + head[u] * sh);
                dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
            }
        }
    }
}

template <int D>
dap_status launch_d(const RunArgs &a, bool write, cudaStream_t stream) {
    const int batch = 4 * 256 / (write ? D / 8 : D / 16);  // rows of a CTA's batch of loads
    const int TT = std::min(kMaxTT, std::max(1, batch / a.Hkv));
    const size_t smem = write ? (size_t)a.Hkv * TT * sizeof(__nv_bfloat16) : 0;
    if (smem > 40 * 1024) return DAP_ERR_UNSUPPORTED;  // (over 20,000 kv heads)
    const dim3 grid((unsigned)((a.T + (long long)TT - 1) / TT), 2);
    const cudaError_t e =
        write ? launch_dependent_smem(append_runs_kernel<D>, grid, dim3(256), (int)smem, stream, a, TT)
              : launch_dependent_smem(read_runs_kernel<D>, grid, dim3(256), 0, stream, a, TT);
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
