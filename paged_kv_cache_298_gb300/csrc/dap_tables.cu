// dap_tables.cu -- the bookkeeping of a paged cache on the GPU: pages taken and returned as the lengths of a batch
// change, with the block table and the slot map that follow from it (kv_resize_paged), and the rows of accepted
// drafted tokens moved to their places (kv_commit_paged).
//
// Resize.  With pages(n) = ceil(n / page_size), sequence b returns pages(old) - pages(new) of its pages, or takes
// pages(new) - pages(old).  R pages are returned in all, A taken.  In order of sequence and entry the r-th returned page
// goes to free_pages[num_free + r], and then the e-th taken entry gets free_pages[num_free + R - A + e]: the stack's top A
// entries, in their order, so that the same step backwards restores the stack.  An entry that is taken from what the call
// itself returns is read from the block table, at its place in the order, not from the stack: no thread waits for
// another's store, and rows of the slot map find their pages the same way.
#include <algorithm>

#include "dap_tile.cuh"

namespace dap {

namespace {

struct ResizeParams {
    const int32_t *old_lens, *new_lens;
    int32_t *block_table;
    int max_pages, page_size, num_pages, B;
    int32_t *free_pages, *num_free;
    int32_t *indptr;
    void *slots;
    int wide, rows;  // 8-byte slots; rows of the slot map
    int rows_here;   // the slot map is written by this kernel (else by slots_kernel)
};

constexpr int kResizeThreads = 512;

// Lengths of sequence b; one out of range leaves its sequence as it is.
struct Lens {
    int from, to;
    bool bad;
};
__device__ __forceinline__ Lens lens_of(const ResizeParams &p, int b) {
    Lens l = {p.old_lens[b], p.new_lens[b], false};
    const long long most = (long long)p.max_pages * p.page_size;
    l.bad = l.from < 0 || l.to < 0 || l.from > most || l.to > most;
    if (l.bad) l.from = l.to = 0;
    return l;
}

__device__ __forceinline__ int pages_of(int n, int ps) { return (int)(((long long)n + ps - 1) / ps); }

// The last i in [0, n) with at[i] <= x (at[0] <= x, ascending).
__device__ __forceinline__ int last_at_most(const int *at, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void store_slot(const ResizeParams &p, long long r, long long slot) {
    if (p.wide) static_cast<int64_t *>(p.slots)[r] = slot;
    else static_cast<int32_t *>(p.slots)[r] = (int32_t)slot;
}

// The slot of position `pos` in page `page`.
__device__ __forceinline__ long long slot_of(const ResizeParams &p, int page, int pos) {
    if (page < 0 || page >= p.num_pages) {
        flag_error(DAP_DEVERR_PAGE);
        return -1;
    }
    return (long long)page * p.page_size + pos % p.page_size;
}

// One cluster.  Every CTA computes the prefix sums of all sequences, and takes its share of the pages and rows; the CTAs
// meet once, before the count of free pages that they all read is replaced.
__global__ void __launch_bounds__(kResizeThreads) resize_kernel(const ResizeParams p) {
    extern __shared__ int smem[];
    int *s_rel = smem, *s_take = smem + (p.B + 1), *s_more = s_take + (p.B + 1);  // exclusive prefix sums, [B + 1]
    __shared__ unsigned long long w_pages[kResizeThreads / 32], w_rows[kResizeThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int count = *p.num_free;
    // (returned << 32 | taken: neither sum passes 2^30, and new rows)
    unsigned long long pages0 = 0, rows0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kResizeThreads) {
        const int b = b0 + tid;
        unsigned long long pages = 0, rows = 0;
        if (b < p.B) {
            const Lens l = lens_of(p, b);
            if (l.bad && blockIdx.x == 0) flag_error(DAP_DEVERR_SEQLEN);
            const int d = pages_of(l.to, p.page_size) - pages_of(l.from, p.page_size);
            pages = d < 0 ? (unsigned long long)(-d) << 32 : (unsigned long long)d;
            rows = (unsigned long long)max(0, l.to - l.from);
        }
        unsigned long long ip = pages, ir = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, ip, o), c = __shfl_up_sync(0xFFFFFFFFu, ir, o);
            if (lane >= o) {
                ip += a;
                ir += c;
            }
        }
        if (lane == 31) {
            w_pages[warp] = ip;
            w_rows[warp] = ir;
        }
        __syncthreads();
        unsigned long long bp = pages0, br = rows0;
        for (int w = 0; w < kResizeThreads / 32; ++w) {
            if (w < warp) {
                bp += w_pages[w];
                br += w_rows[w];
            }
            pages0 += w_pages[w];
            rows0 += w_rows[w];
        }
        if (b < p.B) {
            bp += ip - pages;
            br += ir - rows;
            s_rel[b] = (int)(bp >> 32);
            s_take[b] = (int)(bp & 0xFFFFFFFFu);
            s_more[b] = (int)min(br, 0x7FFFFFFFull);
        }
        __syncthreads();
    }
    const int R = (int)(pages0 >> 32), A = (int)(pages0 & 0xFFFFFFFFu);
    const bool too_long = rows0 > 0x7FFFFFFFull;
    const long long top = (long long)count + R;
    // nothing is changed where the pool cannot give or take the pages
    const bool ok = count >= 0 && count <= p.num_pages && top <= p.num_pages && top - A >= 0 && !too_long;
    const int rows = ok ? (int)rows0 : 0;
    if (tid == 0) {
        s_rel[p.B] = R;
        s_take[p.B] = A;
        s_more[p.B] = rows;
        if (blockIdx.x == 0) {
            if (!ok) flag_error(too_long ? DAP_DEVERR_SEQLEN : DAP_DEVERR_POOL);
            if (rows > p.rows) flag_error(DAP_DEVERR_SLOT);
        }
    }
    // every CTA has read the count
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    const int at = blockIdx.x * kResizeThreads + tid, all = gridDim.x * kResizeThreads;
    if (at == 0 && ok) *p.num_free = (int)(top - A);
    for (int b = at; b <= p.B; b += all) p.indptr[b] = ok ? s_more[b] : 0;
    auto returned = [&](int r) -> int {  // the r-th returned page
        const int b = last_at_most(s_rel, p.B, r);
        const int i = pages_of(lens_of(p, b).to, p.page_size) + r - s_rel[b];
        return p.block_table[(long long)b * p.max_pages + i];
    };
    auto taken = [&](int e) -> int {  // the e-th taken page
        const int i = (int)(top - A) + e;
        return i < count ? p.free_pages[i] : returned(i - count);
    };
    if (ok) {
        for (int r = at; r < R; r += all) p.free_pages[count + r] = returned(r);
        for (int e = at; e < A; e += all) {
            const int b = last_at_most(s_take, p.B, e);
            const int i = pages_of(lens_of(p, b).from, p.page_size) + e - s_take[b];
            p.block_table[(long long)b * p.max_pages + i] = taken(e);
        }
    }
    if (!p.rows_here) return;
    for (int r = at; r < p.rows; r += all) {
        long long slot = -1;
        if (r < rows) {
            const int b = last_at_most(s_more, p.B, r);
            const int from = lens_of(p, b).from, pos = from + r - s_more[b];
            const int i = pos / p.page_size, had = pages_of(from, p.page_size);
            slot = slot_of(p, i < had ? p.block_table[(long long)b * p.max_pages + i] : taken(s_take[b] + i - had), pos);
        }
        store_slot(p, r, slot);
    }
}

// The slot map from the tables and boundaries that resize_kernel wrote.
__global__ void __launch_bounds__(256) slots_kernel(const ResizeParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int rows = p.indptr[p.B];
    for (long long r = (long long)blockIdx.x * 256 + threadIdx.x; r < p.rows; r += (long long)gridDim.x * 256) {
        long long slot = -1;
        if (r < rows) {
            const int b = last_at_most(p.indptr, p.B, (int)r);
            const int pos = p.old_lens[b] + (int)r - p.indptr[b];
            slot = slot_of(p, p.block_table[(long long)b * p.max_pages + pos / p.page_size], pos);
        }
        store_slot(p, r, slot);
    }
}

// ---- accepted drafts ------------------------------------------------------------------------------------------
// The rows of node path[j] go to place j behind the context.  The path ascends strictly, so path[j] >= j, and a place that
// is written is the source of no later row: each thread moves its 16 bytes of every row in order, in place, and no two
// threads share an address.

struct CommitParams {
    uint4 *cache[2];
    int num_pages, page_size, max_pages;
    const int32_t *block_table, *positions, *path, *accepted;
    int max_path, B;
    long long row_chunks;  // 16-byte chunks of a row of all kv heads
    int groups;            // of 32 chunks
};

__global__ void __launch_bounds__(128) commit_kernel(const CommitParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);  // (sequence, K or V, 32 chunks)
    const int lane = threadIdx.x & 31;
    const int per = 2 * p.groups;
    const int b = (int)(w / per), rest = (int)(w - (long long)b * per), x = rest / p.groups;
    if (b >= p.B) return;
    const int n = p.accepted[b];
    const long long base = p.positions[b];
    const int32_t *path = p.path + (long long)b * p.max_path;
    const bool tells = rest == 0 && lane == 0;
    if (n == 0) return;
    // the whole path is looked at before the first row moves
    bool good = n > 0 && n <= p.max_path && base >= 0;
    if (good) {
        bool up = true;
        int last = 0;
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int j = j0 + lane;
            if (j < n) {
                last = path[j];
                up = up && last > (j > 0 ? path[j - 1] : -1);
            }
        }
        good = __all_sync(0xFFFFFFFFu, up);
        if (good) {
            const int end = __shfl_sync(0xFFFFFFFFu, last, (n - 1) & 31);
            if (base + end >= (long long)p.max_pages * p.page_size) {
                if (tells) flag_error(DAP_DEVERR_SEQLEN);
                return;
            }
        }
    }
    if (!good) {
        if (tells) flag_error(base < 0 ? DAP_DEVERR_SEQLEN : DAP_DEVERR_QMAP);
        return;
    }
    const int32_t *table = p.block_table + (long long)b * p.max_pages;
    const long long c = (long long)(rest - x * p.groups) * 32 + lane;
    uint4 *cache = p.cache[x] + c;
    const bool mine = c < p.row_chunks;
    for (int j0 = 0; j0 < n; j0 += 32) {
        // lane j: the cache rows that row j0 + j is read from and goes to; -1: it stays
        long long from = -1, to = -1;
        if (j0 + lane < n) {
            const long long s = base + path[j0 + lane], d = base + j0 + lane;
            if (s != d) {
                const int sp = table[s / p.page_size], dp = table[d / p.page_size];
                if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) {
                    if (rest == 0) flag_error(DAP_DEVERR_PAGE);
                } else {
                    from = (long long)sp * p.page_size + s % p.page_size;
                    to = (long long)dp * p.page_size + d % p.page_size;
                }
            }
        }
        const int m = min(32, n - j0);
        for (int k0 = 0; k0 < m; k0 += 8) {
            uint4 v[8];
            long long at[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const long long f = __shfl_sync(0xFFFFFFFFu, from, (k0 + k) & 31);
                at[k] = __shfl_sync(0xFFFFFFFFu, to, (k0 + k) & 31);
                if (k0 + k >= m) at[k] = -1;
                if (at[k] >= 0 && mine) v[k] = cache[f * p.row_chunks];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (at[k] >= 0 && mine) cache[at[k] * p.row_chunks] = v[k];
        }
    }
}

}  // namespace

dap_status launch_resize(const ResizeArgs &a, cudaStream_t stream) {
    ResizeParams p = {};
    p.old_lens = a.old_lens;
    p.new_lens = a.new_lens;
    p.block_table = a.block_table;
    p.max_pages = a.max_pages;
    p.page_size = a.page_size;
    p.num_pages = a.num_pages;
    p.B = a.B;
    p.free_pages = a.free_pages;
    p.num_free = a.num_free;
    p.indptr = a.indptr;
    p.slots = a.slots;
    p.wide = a.slot_bytes == 8;
    p.rows = a.rows;
    p.rows_here = a.rows <= 8192;
    const int smem = 3 * (a.B + 1) * 4;
    static PerDeviceOcc occ = {};
    if (prepare_kernel(resize_kernel, kResizeThreads, 3 * (kResizeMost + 1) * 4, &occ) <= 0) return DAP_ERR_CUDA;
    const int ctas = a.B > 64 || a.rows > 2048 ? 8 : 1;
    if (launch_cluster_dependent_smem(resize_kernel, dim3((unsigned)ctas), dim3(kResizeThreads), smem, ctas, stream, p) !=
        cudaSuccess)
        return DAP_ERR_CUDA;
    if (p.rows_here) return DAP_OK;
    const dim3 grid((unsigned)std::min(8 * std::max(1, dap_device_sm_count()), (a.rows + 255) / 256));
    return launch_dependent(slots_kernel, grid, dim3(256), stream, p) == cudaSuccess ? DAP_OK : DAP_ERR_CUDA;
}

dap_status launch_commit(const CommitArgs &a, cudaStream_t stream) {
    CommitParams p = {};
    p.cache[0] = static_cast<uint4 *>(a.k_cache);
    p.cache[1] = static_cast<uint4 *>(a.v_cache);
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.max_pages = a.max_pages;
    p.block_table = a.block_table;
    p.positions = a.positions;
    p.path = a.path;
    p.accepted = a.accepted;
    p.max_path = a.max_path;
    p.B = a.B;
    p.row_chunks = (long long)a.Hkv * a.D / 8;
    p.groups = (int)((p.row_chunks + 31) / 32);
    const long long grid = ((long long)a.B * 2 * p.groups + 3) / 4;
    if (grid > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    return launch_dependent(commit_kernel, dim3((unsigned)grid), dim3(128), stream, p) == cudaSuccess ? DAP_OK
                                                                                                      : DAP_ERR_CUDA;
}

bool read_errors_tables(unsigned int *flags, bool clear) {
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
