// dap_shared.cuh -- decode of a batch whose sequences share prefixes: what its kernels have in
// common, and the suffix kernel (instantiated by dap_shared_suffix.cu and, for page sizes that are
// not multiples of 8, dap_shared_suffix_gather.cu).  The prefix kernel is in dap_shared_prefix.cu.
//
// out[b,h] = sum_{t < L_b} softmax_t(scale q[b,h] . K[b,t]) V[b,t], where positions t < P_g hold the
// same keys for every sequence b of group g.  The sum is cut into a prefix part and a suffix part,
// each with its own running maximum and sum:
//   * prefix: the G heads x the sequences of a group are the rows of a matrix product against the
//     group's P_g keys, so every key is read once for up to 256 rows;
//   * suffix: positions P_g .. L_b of each sequence, the split schedule of the single-token decode.
// Each part is cut into splits that leave (acc, m, l) partials in the workspace, [B][prefix splits +
// suffix splits][Hq][D] then [..][2], and a combine kernel merges a row's partials in that order; with one suffix
// split and few prefix partials the suffix kernel does that itself (launch_suffix has the rule).
// The suffix kernel does not wait for the prefix kernel: it starts beside it, on the SMs that the prefix
// leaves free, as soon as every prefix CTA runs (programmatic dependent launch), and one of its CTAs waits
// for the prefix kernel's end before it exits, so that the combine, which waits for the suffix kernel, finds
// both.  The prefix is bound by its products, the suffix by memory: run side by side they use both.  How many
// SMs each gets is a matter of the prefix's split count, which dap_shared_plan chooses for both to end
// together: 64 sequences behind 32768 shared keys, 64 .. 2048 of their own (64 query heads, 8 kv heads, D = 128),
// 96 SMs and 56: 90 us; the prefix on all SMs, then the suffix: 114 us.
// An assumption of that start: the programming model promises a grid sight of earlier grids' writes at its own
// griddepcontrol.wait.  The suffix CTAs and the combine read lengths, tables and K/V without one (the combine: the lengths
// only).  They start after every prefix CTA has passed its wait, so the writers' grids have ended and their writes are in
// L2, and no SM holds older copies, as a grid's start invalidates its L1.  Tested where lengths and K/V are written by the
// call before, again and again without waiting (tests/test_shared_gpu.py: lengths that grow in place, append then
// decode).
#pragma once

#include <algorithm>

#include "dap_decode.cuh"

namespace dap {

struct SharedParams {
    SplitParams sp;  // q, caches, table, lengths, sizes, out; num_splits / chunk are the suffix's
    const int32_t *prefix_lens, *seq_group, *tiles;
    int num_groups, num_tiles, seqs_per_tile, max_prefix_len, max_suffix_len;
    int prefix_splits, prefix_chunk, total_splits;
    int merge;  // the suffix kernel merges and writes the rows (no combine)
    float *o_part, *ml_part;
};

// The prefix length of group g, inside its bound.
__device__ __forceinline__ int group_prefix(const SharedParams &p, int g) {
    return min(max(__ldg(p.prefix_lens + g), 0), p.max_prefix_len);
}

// Prefix length and length of sequence b: a length of 0, below the prefix or of no group means
// that nothing is attended (a zero row).  `flags` gets the error bits.
struct Span {
    int P, L;
};
__device__ __forceinline__ Span seq_span(const SharedParams &p, int b, unsigned int *flags) {
    // (with one group its number need not be read)
    const int g = p.num_groups == 1 ? 0 : __ldg(p.seq_group + b), Lraw = __ldg(p.sp.seq_lens + b);
    if (g < 0 || g >= p.num_groups) {
        *flags |= DAP_DEVERR_QMAP;
        return {0, 0};
    }
    const int Praw = __ldg(p.prefix_lens + g);
    Span s = {min(max(Praw, 0), p.max_prefix_len), Lraw};
    if (Praw != s.P) *flags |= DAP_DEVERR_SEQLEN;
    const long long top =
        min((long long)s.P + p.max_suffix_len, (long long)p.sp.max_pages * p.sp.page_size);
    if (Lraw < 0 || (Lraw > 0 && Lraw < s.P) || Lraw > top) {
        *flags |= DAP_DEVERR_SEQLEN;
        s.L = Lraw < s.P ? 0 : (int)top;
    }
    return s;
}

// Position that the suffix's first tile starts at: the boxes of a page start at multiples of R.
__device__ __forceinline__ int suffix_start(const SharedParams &p, int P) { return P - P % p.sp.box_rows; }
__device__ __forceinline__ int suffix_count(const SharedParams &p, const Span &s) {
    if (s.L <= s.P) return 0;
    return min(p.sp.num_splits, (s.L - suffix_start(p, s.P) + p.sp.chunk - 1) / p.sp.chunk);
}

// Page ids of a producer warp: lane l holds entries base + l and base + 32 + l of the sequence's table row, so that a
// load of 32 entries serves 32 pages and is in flight while the 32 before it are used.  (A page id that was loaded for
// the next tile and range-checked at once held the warp for the load's latency: 0.3 us a tile.)
struct PageWindow {
    const int32_t *row;
    int base, end, lane;
    int cur, nxt;
    __device__ __forceinline__ PageWindow(const int32_t *row_, int first, int max_pages, int lane_)
        : row(row_), base(first), end(max_pages), lane(lane_) {
        cur = get(first + lane);
        nxt = get(first + 32 + lane);
    }
    __device__ __forceinline__ int get(int e) const { return e < end ? __ldg(row + e) : 0; }
    // Entry e of each lane, first <= e < first + 32 (first: the same in every lane, never falling).
    __device__ __forceinline__ int at(int e, int first) {
        if (first >= base + 32) {
            base += 32;
            cur = nxt;
            nxt = get(base + 32 + lane);
        }
        const int a = __shfl_sync(0xFFFFFFFFu, cur, e - base), b = __shfl_sync(0xFFFFFFFFu, nxt, e - base - 32);
        return e - base < 32 ? a : b;
    }
};

// The rows of a row-gather tile by the same window: lane l holds rows l, l + 32, .. of tile after tile, with no
// division after the first.  (A prefix tile at page size 12 against a table read a row: 0.65 us for 0.81 at D = 64,
// 1.27 for 1.35 at D = 256.)
template <class C>
struct RowWalk {
    static constexpr int N = RowPages<C>::N;
    PageWindow pages;
    int e[N], slot[N], first[N], fslot[N];  // entry and slot of the lane's rows, and of row 32 k
    int dq, dr, ps;
    __device__ __forceinline__ RowWalk(const int32_t *row, int tok0, const SplitParams &p, int lane)
        : pages(row, tok0 / p.page_size, p.max_pages, lane), dq(C::BT / p.page_size), dr(C::BT % p.page_size),
          ps(p.page_size) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            first[k] = (tok0 + 32 * k) / ps;
            fslot[k] = (tok0 + 32 * k) % ps;
            e[k] = (tok0 + 32 * k + lane) / ps;
            slot[k] = (tok0 + 32 * k + lane) % ps;
        }
    }
    // The next tile's rows (rows past the tile's end hold anything).
    __device__ __forceinline__ void next(RowPages<C> &rp) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            rp.pg[k] = pages.at(e[k], first[k]);
            rp.slot[k] = slot[k];
            step(e[k], slot[k]);
            step(first[k], fslot[k]);
        }
    }
    __device__ __forceinline__ void step(int &en, int &sl) const {
        en += dq;
        if ((sl += dr) >= ps) {
            sl -= ps;
            ++en;
        }
    }
};

// Row gather of a tile of one tensor, or (BOTH) of K and V behind each other: fill_tile_rows with the source rows of
// eight copies exchanged before the first of them is issued, since a copy's row otherwise costs it the latency of a
// shuffle (a 64-key prefix tile at page size 12: 0.53 us for 0.65 at D = 64, 0.64 for 1.61 at D = 128, 1.00 for 1.27 at
// D = 256).  A row's number fits 32 bits: 2^32 rows of 64 dims are 550 GB.
template <class C, bool BOTH>
__device__ __forceinline__ void gather_rows(uint8_t *tile, const __nv_bfloat16 *x, const __nv_bfloat16 *y,
                                            const RowPages<C> &rp, int nvalid, int kvh, const SplitParams &p,
                                            uint64_t *full, int lane) {
    constexpr int CPR = C::ROWB / 16, N = RowPages<C>::N, RPI = 32 / CPR, U = 8;
    static_assert(C::SWB == 128 && RPI <= 8 && C::BT % (RPI * U) == 0, "batches of whole rows");
    uint32_t row[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int pg = rp.pg[k];
        if (lane + 32 * k < nvalid && (pg < 0 || pg >= p.num_pages)) {
            flag_error(DAP_DEVERR_PAGE);
            pg = 0;
        }
        row[k] = (uint32_t)pg * (uint32_t)p.page_size + (uint32_t)rp.slot[k];
    }
    if (lane == 0) mbar_arrive(full);
    const int c = lane % CPR, r0 = lane / CPR;
    const uint32_t pitch = (uint32_t)(p.Hkv * C::D * 2);
    const uint32_t to = smem_addr(tile) + c / C::CPB * (C::BT * 128) + r0 * 128 + ((c % C::CPB ^ r0) << 4);
    const char *sx = reinterpret_cast<const char *>(x + (long long)kvh * C::D + c * 8);
    const char *sy = BOTH ? reinterpret_cast<const char *>(y + (long long)kvh * C::D + c * 8) : nullptr;
#pragma unroll
    for (int i0 = 0; i0 < C::BT / RPI; i0 += U) {
        uint32_t src[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            src[u] = __shfl_sync(0xFFFFFFFFu, row[(RPI * (i0 + u)) >> 5], (r0 + RPI * (i0 + u)) & 31);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = RPI * (i0 + u);  // (+ r0: the swizzle's chunk is c ^ r0 ^ r's low bits)
            if (r0 + r < nvalid) {
                const uint32_t dst = (to ^ ((r & 7) << 4)) + r * 128;
                const unsigned long long off = (unsigned long long)src[u] * pitch;
                cp_async_16(dst, sx + off);
                if (BOTH) cp_async_16(dst + C::TILE_BYTES, sy + off);
            }
        }
    }
    cp_async_mbar_arrive(full);
}

// ---- suffix kernel: one CTA per (sequence, kv head, split) ---------------------------------------

template <int D_, int G_, bool GATHER_>
struct SuffixCfg {
    // 32-key tiles and two consumer warps, 54 KB: four CTAs share an SM (D = 256: two), so that one's start and end
    // are covered by the others.  128 sequences of 16 .. 1024 keys, D = 128: 42.6 us (0.93 of the copy rate, combine
    // included), against 58 us with 64-key tiles and two CTAs of 107 KB.
    static constexpr int D = D_, G = G_, HG = 1, NWC = 2, BT = 32, NS = D == 64 ? 6 : 3, MINB = D == 256 ? 2 : 4;
    static constexpr bool GATHER = GATHER_, SWZ = true;
    static constexpr int KPW = BT / NWC;
    static constexpr int ROWB = D * 2, SWB = 128, NBLK = ROWB / SWB, CPB = SWB / 16;
    static constexpr int TILE_BYTES = BT * ROWB;
    static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int MRG_OFF = NS * STAGE_BYTES;
    static constexpr int MRG_BYTES = NWC * G * (D / 2 + 2) * 4;
    static constexpr int MISC_OFF = MRG_OFF + MRG_BYTES;
    static constexpr int BAR_OFF = (MISC_OFF + 16 + 7) & ~7;
    static constexpr int SMEM = BAR_OFF + 2 * NS * 8 + 1024;  // + slack to align the base
    static constexpr int THREADS = (NWC + 1) * 32;
    static constexpr int MERGE_NB = shared_merge_batch(G, D);
};

// The prefix partials of the CTA's G heads, merged with its own sums (`sums` + 3 G (D + 2) floats, made by the
// consumers when `mine`): warp w takes partials w, w + 3, ..., then the warps' sums and the suffix's are added.
template <class C>
__device__ __forceinline__ void merge_rows(const SharedParams &pp, float *sums, int b, int kvh, int np, bool mine) {
    constexpr int G = C::G, D = C::D, DPV = D / 32, NB = C::MERGE_NB, W = C::NWC + 1, ROW = D + 2;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row0 = (long long)b * pp.total_splits * p.Hq + kvh * G;
    float M = -INFINITY, l = 0.f, acc[G][DPV];  // (lane: maximum and sum of head lane % G)
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < DPV; ++j) acc[g][j] = 0.f;
    for (int i0 = warp; i0 < np; i0 += NB * W) {
        float x[NB][G][DPV];
        const int own = i0 + W * (lane / G);  // lane k G + g has partial k of head g
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < NB * G && own < np)
            ml = *reinterpret_cast<const float2 *>(pp.ml_part + (row0 + (long long)own * p.Hq + lane % G) * 2);
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (i0 + W * k < np)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    load_row_part<DPV>(pp.o_part + (row0 + (long long)(i0 + W * k) * p.Hq + g) * D + lane * DPV, x[k][g]);
        float m = fmaxf(M, ml.x);
#pragma unroll
        for (int o = G; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float mu = m == -INFINITY ? 0.f : m, old = ex2(M - mu), f = ex2(ml.x - mu);
        float add = f * ml.y;
#pragma unroll
        for (int o = G; o < 32; o <<= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, o);
        M = m;
        l = fmaf(l, old, add);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float og = __shfl_sync(0xFFFFFFFFu, old, g);
#pragma unroll
            for (int j = 0; j < DPV; ++j) acc[g][j] *= og;
        }
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (i0 + W * k < np)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float fg = __shfl_sync(0xFFFFFFFFu, f, k * G + g);
#pragma unroll
                    for (int j = 0; j < DPV; ++j) acc[g][j] = fmaf(fg, x[k][g][j], acc[g][j]);
                }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < DPV; ++j) sums[(warp * G + g) * ROW + lane * DPV + j] = acc[g][j];
    if (lane < G) {
        sums[(warp * G + lane) * ROW + D] = M;
        sums[(warp * G + lane) * ROW + D + 1] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * (D / 2); i += C::THREADS) {
        const int g = i / (D / 2), d = 2 * (i - g * (D / 2));
        float2 v[W + 1], ml[W + 1];
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            const float *from = sums + (k * G + g) * ROW;
            const bool there = k < W || mine;
            v[k] = there ? *reinterpret_cast<const float2 *>(from + d) : make_float2(0.f, 0.f);
            ml[k] = there ? *reinterpret_cast<const float2 *>(from + D) : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, ml[k].x);
        }
        const float mu = m == -INFINITY ? 0.f : m;
        float a0 = 0.f, a1 = 0.f, ls = 0.f;
#pragma unroll
        for (int k = 0; k <= W; ++k) {
            const float f = ex2(ml[k].x - mu);
            a0 = fmaf(f, v[k].x, a0);
            a1 = fmaf(f, v[k].y, a1);
            ls = fmaf(f, ml[k].y, ls);
        }
        store_out_pair(p.out + (long long)b * p.o_sb + (long long)(kvh * G + g) * p.o_sh + d, a0, a1, ls);
    }
}

// The split kernel of dap_decode.cuh with a start position: the same producer and consumer.
template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MINB)
    shared_suffix_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                         const SharedParams pp) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = aligned_smem<C>(smem_raw);
    constexpr int G = C::G, NWC = C::NWC, BT = C::BT, NS = C::NS, D = C::D;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = p.B * p.Hkv;
    const int s = (int)(blockIdx.x / units);
    const int rem = (int)(blockIdx.x - s * units);
    const int b = rem / p.Hkv;
    const int kvh = rem - b * p.Hkv;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *empty = full + NS;
    int *misc = reinterpret_cast<int *>(smem + C::MISC_OFF);  // [0] tiles issued, [1] abort
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], full_arrivals<C>());
            mbar_init(&empty[i], NWC);
        }
        misc[0] = 0;
        misc[1] = 0;
        fence_barrier_init();
    }
    if (!C::GATHER && warp == NWC && lane == 0) {
        prefetch_tensormap(&mapK);
        prefetch_tensormap(&mapV);
    }
    // With a prefix kernel before it, this grid starts once every CTA of that kernel has passed its
    // own wait, so what came before is done (and seen: the assumption above); without one it waits itself.
    if (pp.prefix_splits == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const bool last = pp.prefix_splits > 0 && blockIdx.x == gridDim.x - 1;
    unsigned int flags = 0;
    const Span span = seq_span(pp, b, &flags);  // (flagged by who writes the rows)
    if (pp.merge && flags && kvh == 0 && threadIdx.x == 0) flag_error(flags);
    const int R = p.box_rows, a0 = suffix_start(pp, span.P);
    const int nsplit = suffix_count(pp, span);
    const int tok0 = a0 + s * p.chunk;
    // (the last split takes what the rounding of a0 pushes past the others)
    const int tok1 = s == p.num_splits - 1 ? span.L : min(span.L, tok0 + p.chunk);
    const int ntiles = s < nsplit && tok1 > tok0 ? (tok1 - tok0 + BT - 1) / BT : 0;
    float *sums = reinterpret_cast<float *>(smem);  // (merging, when the ring is idle: [warps + 1][G][D + 2])
    static_assert((NWC + 2) * G * (D + 2) * 4 <= C::MRG_OFF, "the sums fit the ring's place");
    __syncthreads();

    if (ntiles > 0 && warp == NWC) {
        const int32_t *table = p.block_table + (long long)b * p.max_pages;
        int issued = 0;
        if constexpr (C::GATHER) {  // ---- producer warp, row gather
            RowWalk<C> walk(table, tok0, p, lane);
            for (int i = 0; i < ntiles; ++i) {
                const int st = i % NS, t = tok0 + i * BT;
                RowPages<C> rp;
                walk.next(rp);
                if (i >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((i / NS) - 1) & 1))) {
                    misc[1] = 1;
                    break;
                }
                gather_rows<C, true>(smem + st * C::STAGE_BYTES, p.k_cache, p.v_cache, rp, min(BT, tok1 - t), kvh, p,
                                     &full[st], lane);
                issued = i + 1;
            }
        } else {  // ---- producer warp: page lookup + TMA issue
            // (entry and row of box `lane` step from tile to tile, without a division)
            const int dq = BT / p.page_size, dr = BT % p.page_size;
            int e0 = tok0 / p.page_size, row0 = tok0 % p.page_size;  // of the tile's first key
            const int bo = lane * R < BT ? lane * R : 0;
            int idx = (tok0 + bo) / p.page_size, row = (tok0 + bo) % p.page_size;
            PageWindow pages(table, e0, p.max_pages, lane);
            for (int i = 0; i < ntiles; ++i) {
                const int st = i % NS;
                int pg = pages.at(idx, e0);
                if (i >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((i / NS) - 1) & 1))) {
                    misc[1] = 1;
                    break;
                }
                const int nbox = (min(BT, tok1 - (tok0 + i * BT)) + R - 1) / R;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nbox * R * C::ROWB * 2));
                __syncwarp();
                if (lane < nbox) {
                    if (pg < 0 || pg >= p.num_pages) {
                        flag_error(DAP_DEVERR_PAGE);
                        pg = 0;
                    }
                    issue_kv_box<C>(smem + st * C::STAGE_BYTES, lane, R, &mapK, &mapV, kvh, row, pg, &full[st]);
                }
                idx += dq;
                if ((row += dr) >= p.page_size) {
                    row -= p.page_size;
                    ++idx;
                }
                e0 += dq;
                if ((row0 += dr) >= p.page_size) {
                    row0 -= p.page_size;
                    ++e0;
                }
                issued = i + 1;
            }
        }
        if (lane == 0) misc[0] = issued;
    }
    int consumed = 0;
    MmaConsumer<C> cs;
    if (ntiles > 0 && warp < NWC) {  // ---- consumer warps
        cs.init(warp, lane, smem, 31 - __clz(C::GATHER ? BT : R));
        cs.reset();
        cs.load_q(p.q + (long long)b * p.q_sb + (long long)kvh * G * p.q_sh, p.q_sh, p.qscale);
        for (int i = 0; i < ntiles; ++i) {
            const int st = i % NS;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (i / NS) & 1))) {
                misc[1] = 1;
                break;
            }
            cs.template tile<true>(smem + st * C::STAGE_BYTES, min(BT, tok1 - (tok0 + i * BT)),
                                   i == 0 ? span.P - tok0 : 0);
            if (lane == 0) mbar_arrive(&empty[st]);
            consumed = i + 1;
        }
    }
    __syncthreads();  // every consumer is done; the producer has finished issuing
    if (ntiles > 0) {
        if (misc[1]) {  // a wait timed out: drain the copies still in flight (bounded), write nothing
            if (threadIdx.x == 0)
                for (int i = consumed; i < misc[0]; ++i) (void)mbar_wait(&full[i % NS], (i / NS) & 1);
        } else if (warp < NWC) {
            cs.finish(reinterpret_cast<float *>(smem + C::MRG_OFF),
                      [] { named_sync(1, NWC * 32); return true; },
                      [&](int, int g, int d, float a0v, float a1v, float M, float lv) {
                          if (pp.merge) {
                              float *to = sums + ((NWC + 1) * G + g) * (D + 2);
                              to[d] = a0v;
                              to[d + 1] = a1v;
                              if (d == 0) {
                                  to[D] = M;
                                  to[D + 1] = lv;
                              }
                              return;
                          }
                          const long long row =
                              ((long long)b * pp.total_splits + pp.prefix_splits + s) * p.Hq + kvh * G + g;
                          *reinterpret_cast<float2 *>(pp.o_part + row * D + d) = make_float2(a0v, a1v);
                          if (d == 0) *reinterpret_cast<float2 *>(pp.ml_part + row * 2) = make_float2(M, lv);
                      });
        }
    }
    if (last || pp.merge) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (pp.merge && (ntiles == 0 || !misc[1]))
        merge_rows<C>(pp, sums, b, kvh, span.L > 0 ? (span.P + pp.prefix_chunk - 1) / pp.prefix_chunk : 0, ntiles > 0);
}

// ---- host side -------------------------------------------------------------------------------------

// CTAs of the prefix kernel's grid.
inline long long prefix_ctas(const SharedArgs &a) { return (long long)a.num_tiles * a.Hkv * a.prefix_splits; }

namespace {

inline SharedParams shared_params(const SharedArgs &a, int box_rows) {
    SharedParams p = {};
    SplitParams &s = p.sp;
    s.q = static_cast<const __nv_bfloat16 *>(a.q);
    s.q_sb = a.q_sb;
    s.q_sh = a.q_sh;
    s.k_cache = static_cast<const __nv_bfloat16 *>(a.k);
    s.v_cache = static_cast<const __nv_bfloat16 *>(a.v);
    s.block_table = a.block_table;
    s.max_pages = a.max_pages;
    s.seq_lens = a.seq_lens;
    s.B = a.B;
    s.Hq = a.Hq;
    s.Hkv = a.Hkv;
    s.page_size = a.page_size;
    s.num_pages = a.num_pages;
    s.box_rows = box_rows;
    s.num_splits = a.suffix_splits;
    s.chunk = a.suffix_chunk;
    s.qscale = a.scale * 1.4426950408889634f;
    s.out = static_cast<__nv_bfloat16 *>(a.out);
    s.o_sb = a.o_sb;
    s.o_sh = a.o_sh;
    p.prefix_lens = a.prefix_lens;
    p.seq_group = a.seq_group;
    p.tiles = a.tiles;
    p.num_groups = a.num_groups;
    p.num_tiles = a.num_tiles;
    p.seqs_per_tile = a.seqs_per_tile;
    p.max_prefix_len = a.max_prefix_len;
    p.max_suffix_len = a.max_suffix_len;
    p.prefix_splits = a.prefix_splits;
    p.prefix_chunk = a.prefix_chunk;
    p.total_splits = a.prefix_splits + a.suffix_splits;
    p.o_part = static_cast<float *>(a.workspace);
    p.ml_part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) +
                                          partial_acc_bytes(a.B, a.Hq, a.D, p.total_splits));
    return p;
}

// Rows of one TMA box of the suffix's tiles (1: row gather), which also aligns the suffix's start.
inline int suffix_box_rows(const SharedArgs &a) {
    return a.page_size % 8 != 0 ? 1 : gcd_int(a.page_size, 32);
}

template <int D, int G, bool GATHER>
dap_status launch_suffix(const SharedArgs &a, cudaStream_t stream, bool *merged) {
    using C = SuffixCfg<D, G, GATHER>;
    const int R = suffix_box_rows(a);
    CUtensorMap mk = {}, mv = {};
    if (!GATHER && (!encode_cache_map<C>(&mk, a.k, a.D, a.Hkv, a.page_size, a.num_pages, R) ||
                    !encode_cache_map<C>(&mv, a.v, a.D, a.Hkv, a.page_size, a.num_pages, R)))
        return DAP_ERR_CUDA;
    auto kern = shared_suffix_kernel<C>;
    static PerDeviceOcc occ = {};
    const int per_sm = prepare_kernel(kern, C::THREADS, C::SMEM, &occ, 100), sms = dap_device_sm_count();
    if (per_sm <= 0 || sms <= 0) return DAP_ERR_CUDA;
    const long long grid = (long long)a.B * a.Hkv * a.suffix_splits;
    if (grid > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    SharedParams p = shared_params(a, R);
    // With one split a sequence's CTA can merge its rows itself, waiting for the prefix kernel where it is: a launch
    // less (2 us on the host) and a hop less (16 sequences behind 2048 shared keys, 11 prefix partials: 11.0 us for
    // 12.1).  It does where all CTAs are resident beside the prefix's (the wait of the first would hold the others
    // back), and up to two trips to memory for the partials (128 partials of 8 heads x 64: 24.3 us against the
    // combine's 11.9, which has a CTA a row for so many).
    *merged = a.suffix_splits == 1 && a.prefix_splits <= shared_merge_most(G, D) &&
              (a.prefix_splits == 0 || grid <= per_sm * std::max(0LL, sms - prefix_ctas(a)));
    p.merge = *merged;
    return launch_dependent_smem(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, mk, mv, p) ==
                   cudaSuccess
               ? DAP_OK
               : DAP_ERR_CUDA;
}

template <int D, bool GATHER>
dap_status suffix_groups(const SharedArgs &a, cudaStream_t stream, bool *merged) {
    switch (a.Hq / a.Hkv) {
        case 1: return launch_suffix<D, 1, GATHER>(a, stream, merged);
        case 2: return launch_suffix<D, 2, GATHER>(a, stream, merged);
        case 4: return launch_suffix<D, 4, GATHER>(a, stream, merged);
        case 8: return launch_suffix<D, 8, GATHER>(a, stream, merged);
    }
    return DAP_ERR_UNSUPPORTED;
}

template <bool GATHER>
dap_status suffix_dims(const SharedArgs &a, cudaStream_t stream, bool *merged) {
    switch (a.D) {
        case 64: return suffix_groups<64, GATHER>(a, stream, merged);
        case 128: return suffix_groups<128, GATHER>(a, stream, merged);
        case 256: return suffix_groups<256, GATHER>(a, stream, merged);
    }
    return DAP_ERR_UNSUPPORTED;
}

inline bool read_tu_errors(unsigned int *flags, bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_errors, sizeof v) != cudaSuccess) return false;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_device_errors, &z, sizeof z) != cudaSuccess) return false;
    }
    *flags |= v;
    return true;
}

}  // namespace
}  // namespace dap
