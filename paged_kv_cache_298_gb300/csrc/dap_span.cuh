// dap_span.cuh -- attention of new tokens over spans of the paged cache: a sliding window with a few first tokens that
// stay visible (sinks), and trees of drafted tokens, with or without a window.  What its kernels have in common, and the
// warp-level kernel for few query columns, instantiated by dap_span.cu (TMA-fed tiles) and dap_span_gather.cu (page sizes
// that are not multiples of 8).  The kernel for many rows is in dap_span_tc.cu.
//
// Sequence b has n new tokens in places ctx .. ctx + n - 1 of the cache, ctx = L - n.  Token i is at position p_i: ctx + i,
// or, in a tree, ctx + its depth (parents come before their children; the children of the context have depth 0).  It sees
// the places t < ctx and, of the new tokens, those up to itself or, in a tree, its ancestors and itself; with a window w and
// s sinks only those of them whose position is below s or above p_i - w:
//   out_i = sum_t softmax_t(scale q_i . K_t) V_t.
// A tile of new tokens (the packed-q work map of the multi-token decode) therefore reads the places [0, s) and
// [lo, end), where lo is the first that its first token's window has and end lies behind its last token.  The two spans are
// laid behind each other, cut at multiples of a K/V tile, so that a K/V tile has keys of one of them: tile places v below
// s rounded up to tiles are places t = v, those above are t = v + gap.  Splits and chunks are cut in v.  Of the rows between
// s and lo that the rounding leaves in, those of whole copies are not copied, and all enter the products with weight zero and
// V = 0: pages that no token sees are never looked at.
#pragma once

#include "dap_multi.cuh"

namespace dap {

struct SpanParams {
    SplitParams sp;
    const int32_t *parents;
    int window, sinks;
    int gran;  // keys of a K/V tile
};

constexpr int kTreeWords = kTreeMost / 32;

struct SpanTile : MultiTile {
    int ctx;        // places in front of the sequence's new tokens
    int lo;         // first place that the window of the tile's first token has (0: no window)
    int sink_end, gap;  // v -> t
    int len;        // of the spans, in v
    __device__ __forceinline__ int place(int v) const { return v < sink_end ? v : v + gap; }
};

__device__ __forceinline__ bool span_tile(const SpanParams &pp, int b, int tindex, int q0, int q1, int L, int qt,
                                          bool report, SpanTile *t) {
    // (a sequence of length 0 is padding: zero rows, and no error)
    if (!multi_tile(pp.sp, b, tindex, q0, q1, L, qt, report && (L != 0 || b < 0 || b >= pp.sp.B), t)) return false;
    if (pp.parents && t->qlen > kTreeMost) {
        if (report) flag_error(DAP_DEVERR_QMAP);
        return false;
    }
    t->ctx = t->pos0 - t->i0;
    t->lo = pp.window > 0 ? max(0, (pp.parents ? t->ctx : t->pos0) - pp.window + 1) : 0;
    t->sink_end = (pp.sinks + pp.gran - 1) & -pp.gran;
    t->gap = max(0, (t->lo & -pp.gran) - t->sink_end);
    t->len = t->kv_end - t->gap;
    return true;
}

__device__ __forceinline__ int span_splits(const SpanTile &t, int chunk) { return max(1, (t.len + chunk - 1) / chunk); }

// The tree's lines of the tile's tokens: bit j of bits[i] is set where token i of the tile sees node j, depth[i] is
// the token's depth.  `parents` is the sequence's row in shared memory (sanitised: in [-1, own index)).
__device__ __forceinline__ void tree_line(const int *parents, int node, int ctx, int window, int sinks, uint32_t *bits,
                                          int *depth) {
    int d = 0;
    for (int j = parents[node]; j >= 0; j = parents[j]) ++d;
    *depth = d;
    for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
    for (int j = node, e = d; j >= 0; j = parents[j], --e)  // e: depth of j
        if (window == 0 || d - e < window || ctx + e < sinks) bits[j >> 5] |= 1u << (j & 31);
}

// Parents of the sequence's first `n` nodes into shared memory, by `threads` threads.  One that is no earlier node is taken
// for the context (and flagged).
__device__ __forceinline__ void load_parents(int *to, const int32_t *from, int n, int tid, int threads, bool report) {
    for (int i = tid; i < n; i += threads) {
        int x = from[i];
        if (x < -1 || x >= i) {
            if (report) flag_error(DAP_DEVERR_TREE);
            x = -1;
        }
        to[i] = x;
    }
}

// ---- warp-level kernel: 8 NT query columns (tokens x the G heads of a kv head) --------------------------------------
// The multi-token kernel's producer and consumer over spans, in two shapes (launch_span has the rule): KW = 2, 32-key tiles and
// two consumer warps, four CTAs an SM (two at D = 256), so that one's start and end are covered by the others; KW = 4, 64-key
// tiles and four consumer warps, two CTAs an SM (one at D = 256), where there are no more CTAs than that and a tile's chain
// (scores, maximum, weights, values: 0.5 us for 32 keys, 0.7 for 64, D = 128) is what counts (4 sequences of one token behind a
// window of 1024: 9.3 us for 14.0).

template <int D_, int G_, int NT_, int KW_, bool GATHER_>
struct SpanCfg {
    static constexpr bool GATHER = GATHER_, MMA = true, SWZ = true, MASK = false;
    static constexpr int D = D_, G = G_, HG = 1, NT = NT_, CG = 1, KW = KW_, NWC = KW, BT = 16 * KW, KPW = 16;
    static constexpr int NCOL = 8 * NT, QT = NCOL / G;
    static constexpr int NS = D == 32 ? 8 : D == 64 ? (KW == 2 ? 6 : 5) : 3;
    static constexpr int MINB = (D == 256 ? 2 : 4) / (KW / 2);
    static constexpr int ROWB = D * 2, SWB = D >= 64 ? 128 : 64, NBLK = ROWB / SWB, CPB = SWB / 16;
    static constexpr int TILE_BYTES = BT * ROWB, STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int NPART = D == 32 ? 2 : 4;
    static constexpr int MRG_OFF = NS * STAGE_BYTES;
    static constexpr int MRG_BYTES = KW * NCOL * (D / NPART + 2) * 4;
    // a tree's parents (before the merge) and lines
    static constexpr int LINE_OFF = MRG_OFF + (MRG_BYTES > kTreeMost * 4 ? MRG_BYTES : kTreeMost * 4);
    static constexpr int LINE_BYTES = QT * (kTreeWords + 1) * 4;
    static constexpr int MISC_OFF = (LINE_OFF + LINE_BYTES + 15) & ~15;
    static constexpr int BAR_OFF = MISC_OFF + 16;
    static constexpr int SMEM = BAR_OFF + 2 * NS * 8 + 1024;  // + slack to align the base
    static constexpr int THREADS = (NWC + 1) * 32;
    static_assert(NCOL % G == 0 && QT >= 1 && SMEM * MINB <= 227 * 1024 && STAGE_BYTES % 1024 == 0, "span tiling");
};

template <class C>
struct SpanConsumer : MultiConsumer<C> {
    using Base = MultiConsumer<C>;
    using Base::acc;
    using Base::col0;
    using Base::g;
    using Base::key0;
    using Base::l_run;
    using Base::lane;
    using Base::m_run;
    using Base::nq;
    using Base::off;
    using Base::p_base;
    using Base::qb;
    using Base::qscale;
    using Base::rb;
    using Base::t;
    static constexpr int G = C::G, KS = C::D / 16, NT = C::NT;
    int ctx, lo, sinks, lo_last, all_end;  // all_end: places below it are seen by every column that has them in its window
    int lo_col[NT][2];                    // the columns' first places
    const uint32_t *bits;                 // the tile's lines (tree), or NULL

    __device__ __forceinline__ void spans(const SpanParams &pp, const SpanTile &tl, const uint32_t *lines,
                                          const int *depth) {
        bits = pp.parents ? lines : nullptr;
        ctx = tl.ctx;
        lo = tl.lo;
        sinks = pp.sinks;
        all_end = pp.parents ? tl.ctx : tl.pos0 + 1;
        lo_last = pp.window > 0 ? tl.ctx + tl.qlen - pp.window : 0;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int ti = min((col0 + n * 8 + 2 * t + j) / G, tl.ntok - 1);
                lo_col[n][j] = pp.window > 0 ? tl.ctx + (pp.parents ? depth[ti] : tl.i0 + ti) - pp.window + 1 : 0;
            }
    }

    // The 16 keys of this warp in the tile whose first key is at place `at`; `nvalid` of the tile's keys lie before the
    // end of the spans.
    __device__ __forceinline__ void tile(uint8_t *stage, int nvalid, int at) {
        const int nv = nvalid - key0, p0 = at + key0;
        if (nv <= 0) return;
        uint8_t *sV = stage + C::TILE_BYTES;
        // V rows that no column of the tile sees may hold anything: zero them, so that 0 * V stays 0
        const int z0 = max(0, sinks - p0), z1 = lo - p0;  // rows [z0, z1) lie between the spans
        if (nv < 16 || z1 > z0) {
            for (int i = lane; i < 16 * C::NBLK * C::CPB; i += 32) {
                const int r = i / (C::NBLK * C::CPB);
                if (r >= nv || (r >= z0 && r < z1))
                    *reinterpret_cast<uint4 *>(sV + tile_off<C>(key0 + r, i % (C::NBLK * C::CPB), rb)) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
        const uint32_t kbase = smem_addr(stage), vbase = smem_addr(sV);
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[n][j] = 0.f;
        {
            const int key = key0 + (lane & 7) + ((lane >> 3) & 1) * 8;
            const int dcol = ((lane >> 4) & 1) * 8;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a[4];
                ldmatrix_x4(a, kbase + off(key, 16 * k + dcol));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_16816(c[n], a, qb[k][n][0], qb[k][n][1]);
            }
        }
        // every column sees all 16 keys (columns without a token too: they are never written)
        const bool inner = p0 + 16 <= all_end && (p0 >= lo_last || p0 + 16 <= sinks);
        const int k0 = p0 + g, k1 = k0 + 8;
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = __fmul_rn(c[n][j], qscale);  // (rounded once: feeds max and exp)
            if (!inner) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int ti = (col0 + n * 8 + 2 * t + j) / G;
                    auto sees = [&](int k) -> bool {
                        if (ti >= nq) return false;
                        if (bits && k >= ctx) {
                            const int node = k - ctx;
                            return node < kTreeMost && ((bits[ti * kTreeWords + (node >> 5)] >> (node & 31)) & 1u);
                        }
                        return k <= p_base + ti && (k >= lo_col[n][j] || k < sinks);
                    };
                    if (!sees(k0)) s[j] = -INFINITY;
                    if (!sees(k1)) s[j + 2] = -INFINITY;
                }
            }
            float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xFFFFFFFFu, mx[0], o));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xFFFFFFFFu, mx[1], o));
            }
            float alpha[2], mu[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float m_new = fmaxf(m_run[n][j], mx[j]);
                mu[j] = (m_new == -INFINITY) ? 0.f : m_new;
                alpha[j] = ex2(m_run[n][j] - mu[j]);
                m_run[n][j] = m_new;
            }
            const uint32_t w0 = pack_bf16x2(ex2(s[0] - mu[0]), ex2(s[1] - mu[1]));
            const uint32_t w1 = pack_bf16x2(ex2(s[2] - mu[0]), ex2(s[3] - mu[1]));
            // (rounded to V's type for the product; l sums what the product sees)
            const float2 f0 = bf16x2_to_float2(w0), f1 = bf16x2_to_float2(w1);
            l_run[n][0] = l_run[n][0] * alpha[0] + (f0.x + f1.x);
            l_run[n][1] = l_run[n][1] * alpha[1] + (f0.y + f1.y);
            // the running max rarely moves after the first tiles: rescale only when it did
            if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    acc[m][n][0] *= alpha[0];
                    acc[m][n][1] *= alpha[1];
                    acc[m][n][2] *= alpha[0];
                    acc[m][n][3] *= alpha[1];
                }
            }
            b0[n] = movmatrix_trans(w0);
            b1[n] = movmatrix_trans(w1);
        }
        {
            const int key = key0 + (lane & 7) + ((lane >> 4) & 1) * 8;
            const int dcol = ((lane >> 3) & 1) * 8;
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                uint32_t a[4];
                ldmatrix_x4_trans(a, vbase + off(key, 16 * m + dcol));
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16_16816(acc[m][n], a, b0[n], b1[n]);
            }
        }
    }
};

// One CTA per (work tile, kv head, split).
template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MINB)
    span_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV, const SpanParams pp) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = aligned_smem<C>(smem_raw);
    constexpr int G = C::G, NWC = C::NWC, BT = C::BT, NS = C::NS, D = C::D;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int units = p.num_tiles * p.Hkv;
    const int s = blockIdx.x / units;
    const int rem = blockIdx.x - s * units;
    const int w = rem / p.Hkv;
    const int kvh = rem - w * p.Hkv;
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
    // A programmatic dependent of the previous kernel: nothing global is read before the wait.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (no work map: one token per sequence, tile w = sequence w)
    const int wb = p.tile_batch ? p.tile_batch[w] : w, wi = p.tile_index ? p.tile_index[w] : 0;
    const int bb = (wb >= 0 && wb < p.B) ? wb : 0;
    const int q0 = p.qo_indptr ? p.qo_indptr[bb] : bb, q1 = p.qo_indptr ? p.qo_indptr[bb + 1] : bb + 1;
    SpanTile tl;
    const bool first = s == 0 && kvh == 0;
    if (!span_tile(pp, wb, wi, q0, q1, p.seq_lens[bb], C::QT, threadIdx.x == 0 && first, &tl)) return;
    const int nsplit = span_splits(tl, p.chunk);
    if (s >= nsplit) return;
    const int v0 = s * p.chunk, v1 = min(tl.len, v0 + p.chunk);
    const int ntiles = v1 > v0 ? (v1 - v0 + BT - 1) / BT : 0;
    const int R = p.box_rows;
    int *parents = reinterpret_cast<int *>(smem + C::MRG_OFF);
    uint32_t *lines = reinterpret_cast<uint32_t *>(smem + C::LINE_OFF);
    int *depth = reinterpret_cast<int *>(lines + C::QT * kTreeWords);
    __syncthreads();

    if (warp == NWC) {
        const int32_t *table = p.block_table + (long long)tl.b * p.max_pages;
        // places t .. t + rows - 1 lie between the spans: no token of the tile sees them
        auto hidden = [&](int t, int rows) { return t >= pp.sinks && t + rows <= tl.lo; };
        int issued = 0;
        if constexpr (C::GATHER) {  // ---- producer warp, row gather
            RowPages<C> next;
            auto lookup = [&](int i) {
#pragma unroll
                for (int k = 0; k < RowPages<C>::N; ++k) {
                    const int r = lane + 32 * k, v = v0 + i * BT + r, t = tl.place(v0 + i * BT) + r;
                    next.pg[k] = 0;
                    next.slot[k] = 0;
                    if (i < ntiles && v < v1) {  // (a hidden row: some row of a page that is seen)
                        next.pg[k] = table[(hidden(t, 1) ? tl.lo : t) / p.page_size];
                        next.slot[k] = t % p.page_size;
                    }
                }
            };
            lookup(0);
            for (int i = 0; i < ntiles; ++i) {
                const int st = i % NS;
                const RowPages<C> rp = next;
                lookup(i + 1);
                if (i >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((i / NS) - 1) & 1))) {
                    misc[1] = 1;
                    break;
                }
                fill_tile_rows<C>(smem + st * C::STAGE_BYTES, rp, min(BT, v1 - (v0 + i * BT)), kvh, p, 0u, [] {},
                                  &full[st], lane);
                issued = i + 1;
            }
        } else {  // ---- producer warp: page lookup + TMA issue
            // the page of the lane's box, raw (it is looked at a tile later), and whether it has one
            auto lookup = [&](int i, bool *box) -> int {
                const int v = v0 + i * BT + lane * R, t = tl.place(v0 + i * BT) + lane * R;
                *box = i < ntiles && lane * R < BT && v < v1 && !hidden(t, R);
                return *box ? table[t / p.page_size] : 0;
            };
            bool has, has_next;
            int next = lookup(0, &has_next);
            for (int i = 0; i < ntiles; ++i) {
                const int st = i % NS;
                int pg = next;
                has = has_next;
                next = lookup(i + 1, &has_next);
                if (i >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((i / NS) - 1) & 1))) {
                    misc[1] = 1;
                    break;
                }
                const int nbox = __popc(__ballot_sync(0xFFFFFFFFu, has));
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nbox * R * C::ROWB * 2));
                __syncwarp();
                if (has) {
                    if (pg < 0 || pg >= p.num_pages) {
                        flag_error(DAP_DEVERR_PAGE);
                        pg = 0;
                    }
                    issue_kv_box<C>(smem + st * C::STAGE_BYTES, lane, R, &mapK, &mapV, kvh,
                                    (tl.place(v0 + i * BT) + lane * R) % p.page_size, pg, &full[st]);
                }
                issued = i + 1;
            }
        }
        if (lane == 0) misc[0] = issued;
        __syncthreads();
        return;
    }

    // ---- consumer warps
    SpanConsumer<C> cs;
    cs.init(warp, lane, smem, 31 - __clz(C::GATHER ? BT : R));
    cs.reset();
    cs.load_q(p.q + (long long)(tl.q0 + tl.i0) * p.q_sb + (long long)kvh * G * p.q_sh, p.q_sb, p.q_sh, tl.ntok, tl.pos0,
              p.qscale);
    if (pp.parents) {
        load_parents(parents, pp.parents + tl.q0, tl.i0 + tl.ntok, threadIdx.x, NWC * 32, first);
        named_sync(1, NWC * 32);
        if (threadIdx.x < tl.ntok)
            tree_line(parents, tl.i0 + threadIdx.x, tl.ctx, pp.window, pp.sinks, lines + threadIdx.x * kTreeWords,
                      depth + threadIdx.x);
        named_sync(1, NWC * 32);
    }
    cs.spans(pp, tl, lines, depth);
    int consumed = 0;
    for (int i = 0; i < ntiles; ++i) {
        const int st = i % NS;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (i / NS) & 1))) {
            misc[1] = 1;
            break;
        }
        const int v = v0 + i * BT;
        cs.tile(smem + st * C::STAGE_BYTES, min(BT, v1 - v), tl.place(v));
        if (lane == 0) mbar_arrive(&empty[st]);
        consumed = i + 1;
    }
    __syncthreads();
    if (misc[1]) {
        if (threadIdx.x == 0)
            for (int i = consumed; i < misc[0]; ++i) (void)mbar_wait(&full[i % NS], (i / NS) & 1);
        return;
    }
    const bool direct = nsplit == 1;
    const int r0 = tl.q0 + tl.i0;
    cs.finish(reinterpret_cast<float *>(smem + C::MRG_OFF), [] { named_sync(1, NWC * 32); return true; },
              [&](int col, int d, float a0, float a1, float M, float lv) {
                  const long long r = r0 + col / G;
                  const int hq = kvh * G + col % G;
                  if (direct) {
                      store_out_pair(p.out + r * p.o_sb + (long long)hq * p.o_sh + d, a0, a1, lv);
                  } else {
                      const long long row = (r * p.num_splits + s) * p.Hq + hq;
                      *reinterpret_cast<float2 *>(p.o_part + row * D + d) = make_float2(a0, a1);
                      if (d == 0) *reinterpret_cast<float2 *>(p.ml_part + row * 2) = make_float2(M, lv);
                  }
              });
}

// Merge of the split partials of every (token, head) row whose tile took more than one split, as combine_multi_kernel: a
// warp per (token, HPW consecutive heads), SB splits per batch of loads, in split order.
template <int D, int HPW, int SB>
__global__ void __launch_bounds__(256) span_combine_kernel(const SpanParams pp, int qt) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int DPV = D / 32;
    const SplitParams &p = pp.sp;
    const long long gw = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int ngroups = p.Hq / HPW;
    if (gw >= (long long)p.total_q * ngroups) return;
    const int r = (int)(gw / ngroups), hq0 = (int)(gw - (long long)r * ngroups) * HPW;
    int b = r, q0 = r, q1 = r + 1;  // no work map: row r is sequence r's one token
    if (p.qo_indptr) {
        int lo = 0, hi = p.B;  // qo_indptr[lo] <= r < qo_indptr[hi] for a well-formed map
        while (hi - lo > 31) {
            const int step = (hi - lo + 31) >> 5;
            const int x = lo + lane * step;
            const unsigned bal = __ballot_sync(0xFFFFFFFFu, x < hi && p.qo_indptr[x] <= r);
            const int j = bal ? 31 - __clz(bal) : 0;
            lo += j * step;
            hi = min(lo + step, hi);
        }
        const int x = lo + lane;  // entries lo .. hi (hi - lo <= 31, hi <= B)
        const int v = x <= hi ? p.qo_indptr[x] : 0x7FFFFFFF;
        const unsigned bal = __ballot_sync(0xFFFFFFFFu, x < hi && v <= r);
        const int j = bal ? 31 - __clz(bal) : 0;
        q0 = __shfl_sync(0xFFFFFFFFu, v, j);
        q1 = __shfl_sync(0xFFFFFFFFu, v, j + 1);
        b = lo + j;
    }
    SpanTile tl;
    if (!span_tile(pp, b, (r - q0) / qt, q0, q1, p.seq_lens[b], qt, false, &tl)) return;
    const int nsplit = span_splits(tl, p.chunk);
    if (nsplit == 1) return;
    const long long rbase = (long long)r * p.num_splits * p.Hq + hq0;  // row (r, s, hq) = (r S + s) Hq + hq
    float acc[HPW][DPV], lsum[HPW], M[HPW];
#pragma unroll
    for (int h = 0; h < HPW; ++h) {
        lsum[h] = 0.f;
        M[h] = -INFINITY;
#pragma unroll
        for (int j = 0; j < DPV; ++j) acc[h][j] = 0.f;
    }
    for (int s0 = 0; s0 < nsplit; s0 += SB) {
        float x[HPW][SB][DPV];
        float2 ml[HPW][SB];
#pragma unroll
        for (int h = 0; h < HPW; ++h)
#pragma unroll
            for (int k = 0; k < SB; ++k) {
                ml[h][k] = make_float2(-INFINITY, 0.f);
                if (s0 + k < nsplit) {
                    const long long row = rbase + (long long)(s0 + k) * p.Hq + h;
                    load_row_part<DPV>(p.o_part + row * D + lane * DPV, x[h][k]);
                    ml[h][k] = *reinterpret_cast<const float2 *>(p.ml_part + row * 2);
                }
            }
#pragma unroll
        for (int h = 0; h < HPW; ++h) {
            float m = M[h];
#pragma unroll
            for (int k = 0; k < SB; ++k) m = fmaxf(m, ml[h][k].x);
            const float mu = m == -INFINITY ? 0.f : m, old = ex2(M[h] - mu);
            M[h] = m;
            lsum[h] *= old;
#pragma unroll
            for (int j = 0; j < DPV; ++j) acc[h][j] *= old;
#pragma unroll
            for (int k = 0; k < SB; ++k)
                if (s0 + k < nsplit) {
                    const float f = ex2(ml[h][k].x - mu);
                    lsum[h] = fmaf(f, ml[h][k].y, lsum[h]);
#pragma unroll
                    for (int j = 0; j < DPV; ++j) acc[h][j] = fmaf(f, x[h][k][j], acc[h][j]);
                }
        }
    }
#pragma unroll
    for (int h = 0; h < HPW; ++h)
        store_row_part<DPV>(p.out + (long long)r * p.o_sb + (long long)(hq0 + h) * p.o_sh + lane * DPV, acc[h], lsum[h]);
}

namespace {

SpanParams span_params(const SpanArgs &a, int box_rows, int gran) {
    SpanParams p = {};
    p.gran = gran;
    p.sp = make_params(a.d);
    p.sp.box_rows = box_rows;
    p.sp.o_part = static_cast<float *>(a.d.workspace);
    p.sp.ml_part = a.d.num_splits > 1
                       ? reinterpret_cast<float *>(static_cast<char *>(a.d.workspace) +
                                                   partial_acc_bytes(a.d.total_q, a.d.Hq, a.d.D, a.d.num_splits))
                       : nullptr;
    p.parents = a.parents;
    p.window = a.window;
    p.sinks = a.window > 0 ? a.sinks : 0;
    return p;
}

template <int D>
dap_status launch_span_combine(const SpanArgs &a, const SpanParams &p, int qt, cudaStream_t stream) {
    if (a.d.num_splits <= 1) return DAP_OK;
    // Few rows: a warp a row, eight splits a trip to memory, since latency is all there is (one sequence of 8192 keys in 15
    // splits: 17.9 us in all for 26.0); many: four heads a warp, whose sequence is found once.
    const long long rows = (long long)a.d.total_q * a.d.Hq;
    const bool few = rows <= 8192 || a.d.Hq % 4 != 0;
    const long long ctas = ((few ? rows : rows / 4) + 7) / 8;
    if (ctas > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    const dim3 grid((unsigned)ctas);
    const cudaError_t e = few ? launch_dependent(span_combine_kernel<D, 1, 8>, grid, dim3(256), stream, p, qt)
                              : launch_dependent(span_combine_kernel<D, 4, 1>, grid, dim3(256), stream, p, qt);
    return e == cudaSuccess ? DAP_OK : DAP_ERR_CUDA;
}

template <int D, int G, int NT, int KW, bool GATHER>
dap_status launch_span_warp(const SpanArgs &a, cudaStream_t stream) {
    using C = SpanCfg<D, G, NT, KW, GATHER>;
    const int R = GATHER ? 1 : gcd_int(a.d.page_size, C::BT);
    CUtensorMap mk = {}, mv = {};  // (the row-gather producer reads the cache directly)
    if (!GATHER && (!encode_cache_map<C>(&mk, a.d.k, a.d.D, a.d.Hkv, a.d.page_size, a.d.num_pages, R) ||
                    !encode_cache_map<C>(&mv, a.d.v, a.d.D, a.d.Hkv, a.d.page_size, a.d.num_pages, R)))
        return DAP_ERR_CUDA;
    auto kern = span_kernel<C>;
    static PerDeviceOcc occ = {};
    if (prepare_kernel(kern, C::THREADS, C::SMEM, &occ, 100) <= 0) return DAP_ERR_CUDA;
    const long long grid = (long long)a.d.num_tiles * a.d.Hkv * a.d.num_splits;
    if (grid > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    const SpanParams p = span_params(a, R, C::BT);
    if (launch_dependent_smem(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, mk, mv, p) != cudaSuccess)
        return DAP_ERR_CUDA;
    return launch_span_combine<D>(a, p, C::QT, stream);
}

template <int D, int NT, int KW, bool GATHER>
dap_status span_groups(const SpanArgs &a, cudaStream_t stream) {
    switch (a.d.Hq / a.d.Hkv) {
        case 1: return launch_span_warp<D, 1, NT, KW, GATHER>(a, stream);
        case 2: return launch_span_warp<D, 2, NT, KW, GATHER>(a, stream);
        case 4: return launch_span_warp<D, 4, NT, KW, GATHER>(a, stream);
        case 8: return launch_span_warp<D, 8, NT, KW, GATHER>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

// 8 or 16 query columns a tile.
template <int KW, bool GATHER>
dap_status span_dims(const SpanArgs &a, cudaStream_t stream) {
    const bool narrow = a.d.tokens_per_tile * (a.d.Hq / a.d.Hkv) == 8;
    switch (a.d.D) {
        case 32: return narrow ? span_groups<32, 1, KW, GATHER>(a, stream) : span_groups<32, 2, KW, GATHER>(a, stream);
        case 64: return narrow ? span_groups<64, 1, KW, GATHER>(a, stream) : span_groups<64, 2, KW, GATHER>(a, stream);
        case 128: return narrow ? span_groups<128, 1, KW, GATHER>(a, stream) : span_groups<128, 2, KW, GATHER>(a, stream);
        case 256: return narrow ? span_groups<256, 1, KW, GATHER>(a, stream) : span_groups<256, 2, KW, GATHER>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

inline bool read_span_errors(unsigned int *flags, bool clear) {
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
