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
    int part;        // kAll, kNoCount or kCountOnly
    bool vectors;    // the slot map begins at a multiple of 16 bytes
};
enum { kAll, kNoCount, kCountOnly };

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

// (n >= 0; the sum stays below 2^32)
__device__ __forceinline__ int pages_of(int n, int ps) { return (int)(((unsigned)n + (unsigned)ps - 1u) / (unsigned)ps); }

// The last i in [0, n) with at[i] <= x (at[0] <= x, ascending); the same number of steps whatever x, so that several searches
// of a thread run beside each other.
__device__ __forceinline__ int last_at_most(const int *at, int n, int x) {
    int lo = 0;
    for (int step = 1 << (31 - __clz(n)); step > 0; step >>= 1)
        if (lo + step < n && at[lo + step] <= x) lo += step;
    return lo;
}

__device__ __forceinline__ void store_slot(const ResizeParams &p, long long r, long long slot) {
    if (p.wide) static_cast<int64_t *>(p.slots)[r] = slot;
    else static_cast<int32_t *>(p.slots)[r] = (int32_t)slot;
}

// The slot of row `row` of page `page`.
__device__ __forceinline__ long long slot_of(const ResizeParams &p, int page, int row) {
    if (page < 0 || page >= p.num_pages) {
        flag_error(DAP_DEVERR_PAGE);
        return -1;
    }
    return (long long)page * p.page_size + row;
}

// Every CTA computes the prefix sums of all sequences and takes its share of the pages and rows.  All of it in one cluster
// (kAll): the CTAs meet once, before the count of free pages that they all read is replaced.  Many rows: on the whole device
// (kNoCount), and then one CTA for the count (kCountOnly).  LARGE: more than one CTA (one alone gets by with less code, which
// has to come from memory too: 6.0 us for 6.6, 16 sequences of 8 rows taken and returned).
template <bool LARGE>
__global__ void __launch_bounds__(kResizeThreads, 1) resize_kernel(const ResizeParams p) {
    extern __shared__ int smem[];
    // per sequence: exclusive sums of pages returned and taken and of new rows [B + 1]; where its first returned entry is in
    // the block table, less its number, and its first taken one; old length
    int *s_rel = smem, *s_take = s_rel + p.B + 1, *s_more = s_take + p.B + 1, *s_src = s_more + p.B + 1, *s_dst = s_src + p.B + 1;
    int *s_from = s_dst + p.B + 1;
    __shared__ unsigned long long w_pages[kResizeThreads / 32], w_rows[kResizeThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int count = *p.num_free;
    const bool tells = blockIdx.x == 0 && p.part != kCountOnly;
    // (returned << 32 | taken: neither sum passes 2^30; and new rows)
    unsigned long long pages0 = 0, rows0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += kResizeThreads) {
        const int b = b0 + tid;
        unsigned long long pages = 0, rows = 0;
        Lens l = {0, 0, false};
        int had = 0, has = 0;
        if (b < p.B) {
            l = lens_of(p, b);
            if (l.bad && tells) flag_error(DAP_DEVERR_SEQLEN);
            had = pages_of(l.from, p.page_size);
            has = pages_of(l.to, p.page_size);
            pages = has < had ? (unsigned long long)(had - has) << 32 : (unsigned long long)(has - had);
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
        {   // lane w of every warp: the sums of warps 0 .. w
            constexpr int W = kResizeThreads / 32;
            unsigned long long x = lane < W ? w_pages[lane] : 0, y = lane < W ? w_rows[lane] : 0;
#pragma unroll
            for (int o = 1; o < W; o <<= 1) {
                const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, x, o), c = __shfl_up_sync(0xFFFFFFFFu, y, o);
                if (lane >= o) {
                    x += a;
                    y += c;
                }
            }
            const unsigned long long xb = __shfl_sync(0xFFFFFFFFu, x, (warp - 1) & 31), yb = __shfl_sync(0xFFFFFFFFu, y, (warp - 1) & 31);
            if (warp > 0) {
                bp += xb;
                br += yb;
            }
            pages0 += __shfl_sync(0xFFFFFFFFu, x, W - 1);
            rows0 += __shfl_sync(0xFFFFFFFFu, y, W - 1);
        }
        if (b < p.B) {
            bp += ip - pages;
            br += ir - rows;
            s_rel[b] = (int)(bp >> 32);
            s_take[b] = (int)(bp & 0xFFFFFFFFu);
            s_more[b] = (int)min(br, 0x7FFFFFFFull);
            s_src[b] = b * p.max_pages + has - s_rel[b];
            s_dst[b] = b * p.max_pages + had - s_take[b];
            s_from[b] = l.from;
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
        if (tells) {
            if (!ok) flag_error(too_long ? DAP_DEVERR_SEQLEN : DAP_DEVERR_POOL);
            if (rows > p.rows && p.rows > 0) flag_error(DAP_DEVERR_SLOT);
        }
    }
    if (p.part == kAll) {  // every CTA has read the count
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __syncthreads();
    const int at = blockIdx.x * kResizeThreads + tid, all = gridDim.x * kResizeThreads;
    if (at == 0 && ok && p.part != kNoCount) *p.num_free = (int)(top - A);
    if (p.part == kCountOnly) return;
    for (int b = at; b <= p.B; b += all) p.indptr[b] = ok ? s_more[b] : 0;
    auto returned = [&](int r) -> int { return p.block_table[s_src[last_at_most(s_rel, p.B, r)] + r]; };  // the r-th
    auto taken = [&](int e) -> int {  // the e-th taken page
        const int i = (int)(top - A) + e;
        return i < count ? p.free_pages[i] : returned(i - count);
    };
    constexpr int U = 4;  // entries or rows that a thread has in flight
    // The n entries of a list whose sums per sequence are `sums`: next to each other for the lanes of a warp, or, with more of
    // them than one pass takes, U2 in a row for a thread, which then searches for the first alone (75,000 pages taken by the
    // device and returned by one cluster, with 1.2 million rows: 17.4 us for 20.2).
    constexpr int U2 = 8;
    auto entries = [&](const int *sums, int n, auto &&load, auto &&store) {
        if (!LARGE || n <= U * all) {
            for (int e0 = at; e0 < n; e0 += U * all) {
                int x[U], b[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e0 + u * all < n) x[u] = load(e0 + u * all, b[u] = last_at_most(sums, p.B, e0 + u * all));
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e0 + u * all < n) store(e0 + u * all, b[u], x[u]);
            }
            return;
        }
        for (int e0 = U2 * at; e0 < n; e0 += U2 * all) {
            int x[U2], b[U2], i = last_at_most(sums, p.B, e0), end = sums[i + 1];
#pragma unroll
            for (int u = 0; u < U2; ++u) {
                if (e0 + u < n && e0 + u >= end) end = sums[(i = last_at_most(sums, p.B, e0 + u)) + 1];
                b[u] = i;
            }
#pragma unroll
            for (int u = 0; u < U2; ++u)
                if (e0 + u < n) x[u] = load(e0 + u, b[u]);
#pragma unroll
            for (int u = 0; u < U2; ++u)
                if (e0 + u < n) store(e0 + u, b[u], x[u]);
        }
    };
    if (ok) {
        entries(s_rel, R, [&](int r, int b) { return p.block_table[s_src[b] + r]; },
                [&](int r, int, int page) { p.free_pages[count + r] = page; });
        entries(s_take, A, [&](int e, int) { return taken(e); }, [&](int e, int b, int page) { p.block_table[s_dst[b] + e] = page; });
    }
    auto page_of = [&](int b, int i) -> int {  // of entry i of sequence b
        const int e = b * p.max_pages + i - s_dst[b];  // number among the taken; an entry that was there: before them
        return e < s_take[b] ? p.block_table[s_dst[b] + e] : taken(e);
    };
    if (!LARGE || p.part == kAll) {  // a thread's rows far apart: one each, mostly
        for (long long r0 = at; r0 < p.rows; r0 += U * all) {
            long long slot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const long long r = r0 + u * all;
                slot[u] = -1;
                if (r < rows) {
                    const int b = last_at_most(s_more, p.B, (int)r);
                    const int pos = s_from[b] + ((int)r - s_more[b]), i = pos / p.page_size;
                    slot[u] = slot_of(p, page_of(b, i), pos - i * p.page_size);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r0 + u * all < p.rows) store_slot(p, r0 + u * all, slot[u]);
        }
        return;
    }
    // Many rows: U next to each other, which are nearly always of one sequence and one page (1.2 million rows: 20.2 us for 25.8
    // with a search for each; a CTA for 2048 of them instead of 4096: 19.9 for 17.4, of all that happens there and back).
    for (long long r0 = (long long)U * at; r0 < p.rows; r0 += (long long)U * all) {
        long long slot[U];
        int end = 0, left = 0;  // the sequence's last row + 1; rows left in the page
        int b = 0, i = 0;
        long long next = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u;
            slot[u] = -1;
            if (r < rows) {
                if (u == 0 || r >= end || left == 0) {
                    int row = 0;
                    if (u == 0 || r >= end) {
                        b = last_at_most(s_more, p.B, (int)r);
                        end = s_more[b + 1];
                        const int pos = s_from[b] + ((int)r - s_more[b]);
                        i = pos / p.page_size;
                        row = pos - i * p.page_size;
                    } else {
                        ++i;
                    }
                    left = p.page_size - row;
                    next = slot_of(p, page_of(b, i), row);
                }
                slot[u] = next;
                if (next >= 0) ++next;
                --left;
            }
        }
        if (p.vectors && r0 + U <= p.rows) {
            if (p.wide) {
                longlong2 *to = reinterpret_cast<longlong2 *>(static_cast<int64_t *>(p.slots) + r0);
                to[0] = make_longlong2(slot[0], slot[1]);
                to[1] = make_longlong2(slot[2], slot[3]);
            } else {
                *reinterpret_cast<int4 *>(static_cast<int32_t *>(p.slots) + r0) =
                    make_int4((int)slot[0], (int)slot[1], (int)slot[2], (int)slot[3]);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r0 + u < p.rows) store_slot(p, r0 + u, slot[u]);
        }
    }
}

// ---- accepted drafts ------------------------------------------------------------------------------------------
// The rows of node path[j] go to place j behind the context.  The path ascends strictly, so path[j] >= j: with 32 rows at a
// time read before any of them is written, no place that is written is the source of a later batch, and pieces of a row are
// independent.  One warp moves a piece of up to 1 KB of every row of a sequence's path, K or V: a lane a row, by bulk copies
// through shared memory, so that all rows of a batch are in flight at once whatever the registers (7.8 us for 15.8 with
// 16-byte loads, 16 rows in flight: 256 paths of up to 24 rows of 2 KB).

struct CommitParams {
    char *k_cache, *v_cache;
    int num_pages, page_size, max_pages;
    const int32_t *block_table, *positions, *path, *accepted;
    int max_path, row_bytes, pieces;
};
constexpr int kPieceBytes = 1024;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}

__global__ void __launch_bounds__(32) commit_kernel(const CommitParams p) {
    __shared__ __align__(128) char rows[32 * kPieceBytes];
    __shared__ uint64_t bar;
    const int lane = threadIdx.x;
    const int b = blockIdx.x / (2 * p.pieces), rest = blockIdx.x - b * 2 * p.pieces;  // (sequence, K or V, piece)
    const int at = (rest >> 1) * kPieceBytes, bytes = min(kPieceBytes, p.row_bytes - at);
    if (lane == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t *path = p.path + (long long)b * p.max_path;
    // (one trip for all three: the first 32 nodes are there whatever the count)
    const int n = p.accepted[b], head = lane < p.max_path ? path[lane] : 0;
    const long long base = p.positions[b];
    const bool tells = rest == 0 && lane == 0;
    if (n == 0) return;
    // the whole path is looked at before the first row moves
    bool good = n > 0 && n <= p.max_path && base >= 0;
    if (good) {
        bool up = true;
        int last = -1;  // the node before lane 0's, then the path's last
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int j = j0 + lane, x = j0 == 0 ? head : j < n ? path[j] : 0;
            const int left = __shfl_up_sync(0xFFFFFFFFu, x, 1);
            if (j < n) up = up && x > (lane > 0 ? left : last);
            last = __shfl_sync(0xFFFFFFFFu, x, min(31, n - 1 - j0));
        }
        good = __all_sync(0xFFFFFFFFu, up);
        if (good && base + last >= (long long)p.max_pages * p.page_size) {
            if (tells) flag_error(DAP_DEVERR_SEQLEN);
            return;
        }
    }
    if (!good) {
        if (tells) flag_error(base < 0 ? DAP_DEVERR_SEQLEN : DAP_DEVERR_QMAP);
        return;
    }
    const int32_t *table = p.block_table + (long long)b * p.max_pages;
    char *cache = ((rest & 1) ? p.v_cache : p.k_cache) + at, *mine = rows + lane * kPieceBytes;
    const uint32_t ps = p.page_size;
    uint32_t phase = 0;
    for (int j0 = 0; j0 < n; j0 += 32) {
        // lane j: the cache rows that row j0 + j is read from and goes to (places are below 2^31 + 2^31)
        long long from = 0, to = -1;  // (-1: it stays)
        if (j0 + lane < n) {
            const uint32_t s = (uint32_t)(base + (j0 == 0 ? head : path[j0 + lane])), d = (uint32_t)(base + j0 + lane);
            if (s != d) {
                const uint32_t se = s / ps, de = d / ps;
                const int sp = table[se], dp = table[de];
                if (sp < 0 || sp >= p.num_pages || dp < 0 || dp >= p.num_pages) {
                    if (rest == 0) flag_error(DAP_DEVERR_PAGE);
                } else {
                    from = (long long)sp * ps + (s - se * ps);
                    to = (long long)dp * ps + (d - de * ps);
                }
            }
        }
        const uint32_t moves = __ballot_sync(0xFFFFFFFFu, to >= 0);
        if (moves == 0) continue;
        if (lane == 0) mbar_arrive_expect_tx(&bar, (uint32_t)__popc(moves) * (uint32_t)bytes);
        __syncwarp();
        if (to >= 0) bulk_load(mine, cache + from * p.row_bytes, (uint32_t)bytes, &bar);
        // (a phase a batch that moves anything)
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar, phase))) {
            (void)mbar_wait(&bar, phase);  // gave up: once more for the copies in flight, before the shared memory goes
            return;
        }
        phase ^= 1u;
        if (to >= 0) bulk_store(cache + to * p.row_bytes, mine, (uint32_t)bytes);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
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
    p.vectors = (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0;
    const int smem = 6 * (a.B + 1) * 4;
    constexpr int kMostSmem = 6 * (kResizeMost + 1) * 4;
    const bool large = a.B > 64 || a.rows > 2048;
    static PerDeviceOcc occ[2] = {};
    if (prepare_kernel(large ? resize_kernel<true> : resize_kernel<false>, kResizeThreads, kMostSmem, &occ[large]) <= 0)
        return DAP_ERR_CUDA;
    // One cluster while its threads have up to four rows each, else the whole device and a launch for the count (1.2 million
    // rows on 256 sequences taken and returned: 17.4 us, with the pages by a cluster 48); one CTA where that is enough (16
    // sequences of 8 rows: 3.0 us).
    constexpr int kClusterRows = 4 * 8 * kResizeThreads;
    if (a.rows <= kClusterRows) {
        p.part = kAll;
        return launch_cluster_dependent_smem(large ? resize_kernel<true> : resize_kernel<false>, dim3(large ? 8u : 1u),
                                             dim3(kResizeThreads), smem, large ? 8 : 1, stream, p) == cudaSuccess
                   ? DAP_OK
                   : DAP_ERR_CUDA;
    }
    const int most = std::max(1, dap_device_sm_count()) * (smem <= 48 * 1024 ? 4 : 1);
    const int ctas = (int)std::min<long long>(most, (a.rows + 8LL * kResizeThreads - 1) / (8 * kResizeThreads));
    p.part = kNoCount;
    if (launch_dependent_smem(resize_kernel<true>, dim3((unsigned)ctas), dim3(kResizeThreads), smem, stream, p) != cudaSuccess)
        return DAP_ERR_CUDA;
    p.part = kCountOnly;
    return launch_dependent_smem(resize_kernel<true>, dim3(1), dim3(kResizeThreads), smem, stream, p) == cudaSuccess ? DAP_OK
                                                                                                                    : DAP_ERR_CUDA;
}

dap_status launch_commit(const CommitArgs &a, cudaStream_t stream) {
    CommitParams p = {};
    p.k_cache = static_cast<char *>(a.k_cache);
    p.v_cache = static_cast<char *>(a.v_cache);
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.max_pages = a.max_pages;
    p.block_table = a.block_table;
    p.positions = a.positions;
    p.path = a.path;
    p.accepted = a.accepted;
    p.max_path = a.max_path;
    const long long row_bytes = (long long)a.Hkv * a.D * 2, pieces = (row_bytes + kPieceBytes - 1) / kPieceBytes;
    if (row_bytes > 0x7FFFFFFFLL || 2 * pieces * a.B > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    p.row_bytes = (int)row_bytes;
    p.pieces = (int)pieces;
    return launch_dependent(commit_kernel, dim3((unsigned)(2 * pieces * a.B)), dim3(32), stream, p) == cudaSuccess
               ? DAP_OK
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
