// dap_span_tc.cu -- attention over spans of the paged cache (dap_span.cuh has the operation) for many query rows, on the
// tcgen05 tensor cores: verification of larger trees, chunks of prompts behind a window.
//
// One CTA takes a work tile of up to 256 query rows of one kv head (row r: new token r / G of the tile, head r % G), or 128
// at D = 256, against one chunk of the tile's spans, in two streams of 128 rows (one at D = 256), as the prefix kernel of
// the shared-prefix decode does (dap_shared_prefix.cu; the ring, the two score buffers a stream, who issues what and why
// are described there): with more than 128 rows each stream has its own and both take every K/V tile of 64 keys, else both
// hold the same rows and take every other tile, merged through shared memory at the end.  What differs:
//   * the tiles walk two spans (the sinks, the window), and a tile has to be masked by row where an end of a window, the
//     new tokens or a tree's nodes lie in it.  A row's mask of the 64 keys is one 64-bit word, made of its bounds and its
//     line of ancestors; tiles that every row of a warp sees whole, nearly all, skip it;
//   * V rows that no row of the tile sees are zeroed by the softmax threads, before they hand over the tile's weights;
//   * with one split the rows leave as bf16 outputs, whole rows a store, and no combine follows.
#include <algorithm>

#include "dap_span.cuh"
#include "dap_tc.cuh"

namespace dap {

namespace {

template <int D_, bool GATHER_>
struct SpanTcCfg {
    static constexpr bool GATHER = GATHER_, SWZ = true;
    static constexpr int D = D_, BT = 64;
    static constexpr int ROWB = D * 2, SWB = 128, NBLK = ROWB / SWB, CPB = SWB / 16;
    static constexpr int TILE_BYTES = BT * ROWB;  // K or V of one tile
    static constexpr int NSTREAM = D == 256 ? 1 : 2, ROWS = 128 * NSTREAM;
    static constexpr int NS = D == 64 ? 6 : D == 128 ? 4 : 2;  // K/V tiles in the ring
    static constexpr int NWS = 4 * NSTREAM, PRODUCER = NWS, ISSUER = NWS + 2, PV = ISSUER + NSTREAM,
                         THREADS = (PV + 1) * 32;
    static constexpr int TO = 256, TMEM_COLS = 512;
    static constexpr int QBLK = 128 * 128, Q_BYTES = NSTREAM * NBLK * QBLK;  // 64 dims of 128 rows; all of q
    static constexpr int RING_OFF = Q_BYTES, BAR_OFF = RING_OFF + NS * 2 * TILE_BYTES;
    // barriers: k_full, k_empty, v_full, v_empty [NS], s_done, p_ready, pv_done [stream][buffer], q_full, fin[3]
    static constexpr int NBAR = 4 * NS + 16;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    // a tree's parents, lines and depths (G = 1: as many tokens as rows)
    static constexpr int TREE_OFF = MISC_OFF + 32, LINE_OFF = TREE_OFF + kTreeMost * 4;
    static constexpr int SMEM = LINE_OFF + ROWS * (kTreeWords + 1) * 4 + 1024;  // + slack to align the base
    static constexpr int ROW_F = D + 4;  // floats of a row of sums on its way out (the 4: no bank conflicts)
    static_assert(SMEM > 114 * 1024 && SMEM <= 227 * 1024, "one CTA an SM: a second would wait for tensor memory");
    static_assert(ROWS * ROW_F * 4 <= BAR_OFF, "the sums on their way out fit the place of q and the ring");
};

// A row's place among a warp's 32 rows of sums, ROW_F floats apart in shared memory, to global memory: `n` rows, NC of their
// floats from `out` + the lane's `to` on, as they are or, with BF16, times the lane's `inv` and rounded.  Whole rows a
// store, eight stores' loads ahead of the first.
template <class C, int NC, bool BF16>
__device__ __forceinline__ void leave(const float *rows, void *out, long long to, float inv, int n, int lane) {
    constexpr int PER = BF16 ? 8 : 4, W = NC / PER < 32 ? NC : 32 * PER, LPR = W / PER, RPI = 32 / LPR, U = 4;
    static_assert(NC % W == 0 && 32 % (RPI * U) == 0, "whole batches");
    __syncwarp();
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += W) {
        const int c = c0 + lane % LPR * PER;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += RPI * U) {
            uint4 v[U];
            long long at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * RPI + lane / LPR;
                at[u] = __shfl_sync(0xFFFFFFFFu, to, i & 31);
                const float f = BF16 ? __shfl_sync(0xFFFFFFFFu, inv, i & 31) : 1.f;
                const float4 x = *reinterpret_cast<const float4 *>(rows + i * C::ROW_F + c);
                if constexpr (BF16) {
                    const float4 y = *reinterpret_cast<const float4 *>(rows + i * C::ROW_F + c + 4);
                    v[u] = make_uint4(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f),
                                      pack_bf16x2(y.x * f, y.y * f), pack_bf16x2(y.z * f, y.w * f));
                } else {
                    v[u] = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                                      __float_as_uint(x.w));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * RPI + lane / LPR < n) {
                    if constexpr (BF16) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + at[u] + c) = v[u];
                    else *reinterpret_cast<uint4 *>(static_cast<float *>(out) + at[u] + c) = v[u];
                }
        }
    }
}

// The n lowest of 64 bits.
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Bits o .. o + 63 of a line (o > -64; what lies outside the line is 0).
__device__ __forceinline__ uint64_t line_bits(const uint32_t *line, int o) {
    auto word = [&](int w) -> uint64_t { return w >= 0 && w < kTreeWords ? line[w] : 0u; };
    const int w = o >> 5, sh = o & 31;
    const uint64_t x = word(w) | word(w + 1) << 32;
    return sh ? x >> sh | word(w + 2) << (64 - sh) : x;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    span_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, const SpanParams pp, const int G) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = aligned_smem<C>(smem_raw);
    constexpr int BT = C::BT, NS = C::NS, D = C::D;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
    uint64_t *s_done = v_empty + NS, *p_ready = s_done + 4, *pv_done = p_ready + 4;  // [2 stream + buffer]
    uint64_t *q_full = pv_done + 4, *fin = q_full + 1;
    // [0], [1] K and V tiles issued, [2] abort, [4] tensor memory
    volatile int *misc = reinterpret_cast<volatile int *>(smem + C::MISC_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF) + 4;
    uint8_t *ring = smem + C::RING_OFF;

    const int units = p.num_tiles * p.Hkv;
    const int s = (int)(blockIdx.x / units);
    const int rem = (int)(blockIdx.x - s * units);
    const int w = rem / p.Hkv;
    const int kvh = rem - w * p.Hkv;

    // Tensor memory touches nothing the previous kernel writes: it is allocated before the wait.
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == C::PRODUCER && lane == 0) {
        prefetch_tensormap(&mapQ);
        if (!C::GATHER) {
            prefetch_tensormap(&mapK);
            prefetch_tensormap(&mapV);
        }
    }
    // Nothing global is read before the wait; the next kernels may start once every CTA holds its tensor memory (they may
    // take some before they wait for this one).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int wb = p.tile_batch[w], wi = p.tile_index[w];
    const int bb = (wb >= 0 && wb < p.B) ? wb : 0;
    const int qt = C::ROWS / G;
    SpanTile tl;
    const bool first = s == 0 && kvh == 0;
    const bool live = span_tile(pp, wb, wi, p.qo_indptr[bb], p.qo_indptr[bb + 1], p.seq_lens[bb], qt,
                                threadIdx.x == 0 && first, &tl);
    const int nsplit = live ? span_splits(tl, p.chunk) : 0;
    const int nrows = s < nsplit ? tl.ntok * G : 0;
    const int v0 = s * p.chunk, v1 = s < nsplit ? min(tl.len, v0 + p.chunk) : v0;
    const int J = max(0, v1 - v0 + BT - 1) / BT;  // K/V tiles of this CTA
    const bool work = nrows > 0 && J > 0;
    const bool both = C::NSTREAM == 2 && nrows > 128;  // the streams have rows of their own
    // K/V tiles of stream x: all of them, or tiles x, x + 2, ...
    auto tiles_of = [&](int x) { return both || C::NSTREAM == 1 ? J : (J - x + 1) / 2; };
    auto tile_at = [&](int x, int n) { return both || C::NSTREAM == 1 ? n : 2 * n + x; };
    auto rows_of = [&](int x) { return both ? min(128, nrows - 128 * x) : nrows; };
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&k_full[i], full_arrivals<C>());
            mbar_init(&v_full[i], full_arrivals<C>());
            // a commit of every stream that takes the K tile, one after the last product that reads the V tile
            mbar_init(&k_empty[i], both ? 2 : 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int e = 0; e < 4; ++e) {
            mbar_init(&s_done[e], 1);
            mbar_init(&p_ready[e], (uint32_t)max(1, (rows_of(e >> 1) + 31) / 32));  // one per warp with rows
            mbar_init(&pv_done[e], 1);
        }
        mbar_init(q_full, 1);
        for (int i = 0; i < 3; ++i) mbar_init(&fin[i], 1);
        misc[0] = misc[1] = misc[2] = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();  // barriers and the tensor-memory address are visible
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t CS = BT * 128;  // bytes between column blocks of a tile
    constexpr uint32_t idS = idesc_bf16(128, BT, 0), idO = idesc_bf16(128, D, 1);
    const int nlast = v1 - (v0 + (J - 1) * BT);  // keys of the last tile

    if (work && (warp == C::PRODUCER || warp == C::PRODUCER + 1)) {
        // ---- a producer warp each for K and V
        const int tensor = warp - C::PRODUCER;
        const int32_t *table = p.block_table + (long long)tl.b * p.max_pages;
        const int R = p.box_rows;
        uint64_t *full = tensor ? v_full : k_full, *empty = tensor ? v_empty : k_empty;
        uint8_t *place = ring + tensor * C::TILE_BYTES;
        int done = 0;  // tiles issued
        auto load_q = [&] {  // 64 dims of 128 rows a copy (rows past the tile's tokens are never read)
            if (tensor == 0 && lane == 0) {
                const int parts = both ? 2 : 1;
                mbar_arrive_expect_tx(q_full, (uint32_t)(parts * C::NBLK * C::QBLK));
                for (int x = 0; x < parts; ++x)
                    for (int cb = 0; cb < C::NBLK; ++cb)
                        tma_load_3d(smem + (x * C::NBLK + cb) * C::QBLK, &mapQ, cb * 64, kvh * G,
                                    tl.q0 + tl.i0 + x * (128 / G), q_full);
            }
            __syncwarp();
        };
        // places t .. t + rows - 1 lie between the spans: no token of the tile sees them
        auto hidden = [&](int t, int rows) { return t >= pp.sinks && t + rows <= tl.lo; };
        if constexpr (C::GATHER) {
            RowPages<C> next;
            auto lookup = [&](int i) {  // (raw ids: they are looked at a tile later)
#pragma unroll
                for (int k = 0; k < RowPages<C>::N; ++k) {
                    const int r = lane + 32 * k, v = v0 + i * BT, t = tl.place(v) + r;
                    next.pg[k] = 0;
                    next.slot[k] = 0;
                    if (i < J && v + r < v1) {
                        next.pg[k] = __ldg(table + (hidden(t, 1) ? tl.lo : t) / p.page_size);
                        next.slot[k] = t % p.page_size;
                    }
                }
            };
            lookup(0);
            load_q();
            for (; done < J; ++done) {
                const int st = done % NS;
                const RowPages<C> rp = next;
                lookup(done + 1);
                if (done >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((done / NS) - 1) & 1))) break;
                gather_rows<C, false>(place + st * 2 * C::TILE_BYTES, tensor ? p.v_cache : p.k_cache, nullptr, rp,
                                      min(BT, v1 - (v0 + done * BT)), kvh, p, &full[st], lane);
            }
        } else {
            // K: lane = (box j, column block cb), or a whole tile where a page has one; V: lane = box, all blocks.  A
            // lane steps the entry and the row of its box from tile to tile (no division but at a span's start).
            const CUtensorMap *map = tensor ? &mapV : &mapK;
            const int kb = tensor || R == BT ? 1 : C::NBLK;
            const int j = lane / kb, cb = lane % kb;
            const int to = tensor ? j * R * C::ROWB : cb * (int)CS + j * R * 128;
            const int dq = BT / p.page_size, dr = BT - dq * p.page_size;
            int e0, row0, e, row;  // of the tile's first place and of the lane's box
            auto start = [&](int t) {
                e0 = t / p.page_size;
                row0 = t - e0 * p.page_size;
                e = e0;
                row = row0 + (j * R < BT ? j * R : 0);  // (lanes without a box follow the tile's first)
                for (; row >= p.page_size; ++e) row -= p.page_size;
            };
            auto ahead = [&](int &en, int &ro) {
                en += dq;
                if ((ro += dr) >= p.page_size) {
                    ro -= p.page_size;
                    ++en;
                }
            };
            start(tl.place(v0));
            PageWindow pages(table, e0, p.max_pages, lane);
            // (the window's first entries are asked for before the sinks' tiles)
            const bool jumps = tl.gap > 0 && v0 < tl.s64 && tl.s64 < v1;
            PageWindow beyond(table, jumps ? tl.place(tl.s64) / p.page_size : e0, p.max_pages, lane);
            const int shown = __ldg(table + tl.lo / p.page_size);
            load_q();
            for (; done < J; ++done) {
                const int st = done % NS, v = v0 + done * BT, t = tl.place(v);
                if (jumps && v == tl.s64) {
                    start(t);
                    pages = beyond;
                }
                const int nbox = (min(BT, v1 - v) + R - 1) / R;
                int pg = pages.at(e, e0);
                if (hidden(t + j * R, R)) pg = shown;
                if (done >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((done / NS) - 1) & 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(nbox * R * C::ROWB));
                __syncwarp();
                if (j < nbox) {
                    if (pg < 0 || pg >= p.num_pages) {
                        flag_error(DAP_DEVERR_PAGE);
                        pg = 0;
                    }
                    tma_load_5d(place + st * 2 * C::TILE_BYTES + to, map, 0, row, cb, kvh, pg, &full[st]);
                }
                ahead(e, row);
                ahead(e0, row0);
            }
        }
        if (done < J) misc[2] = 1;
        if (lane == 0) misc[tensor] = done;
        __syncwarp();
        // every commit on these barriers has arrived before the CTA ends
        for (int i = max(0, J - NS); i < J && done == J; ++i)
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[i % NS], (i / NS) & 1))) {
                misc[2] = 1;
                break;
            }
    } else if (work && warp >= C::ISSUER) {
        // ---- issuing warps: one a stream for its scores, one for all products with V.  The whole warp runs its loop with
        // values that are the same in every lane (and known to be), one lane issues: descriptors then stay in uniform
        // registers.  Two barriers are polled at a time, each by half the lanes.
        auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
        const int role = same(warp - C::ISSUER);  // a stream's scores; NSTREAM: all products with V
        const int Ju = same(J), last = same(nlast);
        const bool two = same(both) != 0;
        const uint32_t tm = same(tmem);
        const int step = two || C::NSTREAM == 1 ? 1 : 2;  // tile n of stream x is step * n + (step == 2 ? x : 0)
        const uint32_t sQ = smem_addr(smem), sR = smem_addr(ring);
        // A V tile is made of boxes [column block][vR keys][128 bytes]; byte offset of key 16 i and the strides of
        // the product's blocks of 64 dims and groups of 8 keys.
        const int vR = same(p.box_rows);
        const uint32_t v_lbo = vR * 128, v_sbo = vR == 8 ? 8 * C::ROWB : 1024;
        auto v_off = [&](int i) -> uint32_t { return i * 16 / vR * vR * C::ROWB + i * 16 % vR * 128; };
        const uint32_t a1 = v_off(1) >> 4, a2 = v_off(2) >> 4, a3 = v_off(3) >> 4;
        auto wait = [&](uint64_t *b0, int n0, uint64_t *b1, int n1) -> bool {
            const bool odd = lane & 1;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(odd ? b1 : b0, (odd ? n1 : n0) & 1)) != 0;
            if (C::GATHER) fence_async_smem();  // (K and V rows were copied by the generic proxy)
            tc_fence_after();
            return ok;
        };
        auto scores = [&](int x, int n) -> bool {
            const int j = step * n + (step == 2 ? x : 0), st = j % NS, e = 2 * x + (n & 1);
            uint64_t *k = &k_full[st];
            if (!(n >= 2 ? wait(k, j / NS, &pv_done[e], (n - 2) >> 1) : wait(k, j / NS, q_full, 0))) return false;
            const uint64_t dQ = sw128_desc(sQ + (two ? x * C::NBLK * C::QBLK : 0), 16, 1024);
            const uint64_t dK = sw128_desc(sR + st * 2 * C::TILE_BYTES, 16, 1024);
            const uint32_t tS = tm + 64 * e;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    umma_bf16(tS, dQ + (((i >> 2) * C::QBLK + (i & 3) * 32) >> 4),
                              dK + (((i >> 2) * CS + (i & 3) * 32) >> 4), idS, i > 0);
                umma_commit(&s_done[e]);
                umma_commit(&k_empty[st]);
            }
            __syncwarp();
            return true;
        };
        auto values = [&](int x, int n) -> bool {
            const int j = step * n + (step == 2 ? x : 0), st = j % NS, e = 2 * x + (n & 1);
            if (!wait(&p_ready[e], n >> 1, &v_full[st], j / NS)) return false;
            const int nv = j == Ju - 1 ? last : BT;
            const uint64_t dV = sw128_desc(sR + (st * 2 + 1) * C::TILE_BYTES, v_lbo, v_sbo);
            const uint32_t tP = tm + 64 * e, tOx = tm + C::TO + x * D;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < BT / 16; ++i)
                    if (i * 16 < nv)
                        umma_bf16_tmem_a(tOx, tP + i * 8, dV + (i == 0 ? 0u : i == 1 ? a1 : i == 2 ? a2 : a3), idO,
                                         n > 0 || i > 0);
                umma_commit(&pv_done[e]);
                if (!two || x == 1) umma_commit(&v_empty[st]);  // (a commit covers all products before it)
            }
            __syncwarp();
            return true;
        };
        const int N0 = (Ju + step - 1) / step, N1 = C::NSTREAM == 1 ? 0 : Ju / step;
        bool ok = true;
        if (role == C::NSTREAM) {
            for (int n = 0; ok && n < N0; ++n) ok = values(0, n) && (n >= N1 || values(1, n));
        } else {
            for (int n = 0; ok && n < (role == 0 ? N0 : N1); ++n) ok = scores(role, n);
        }
        if (!ok && lane == 0) misc[2] = 1;
        if (elect_one()) umma_commit(&fin[role]);  // this warp's products are done when it completes
        __syncwarp();
    }

    // ---- softmax warps: thread = row of a stream
    const int x = warp >> 2;  // stream (warps below NWS)
    const int r = threadIdx.x & 127;
    const bool soft = work && warp < C::NWS;
    const int nx = soft ? rows_of(x) : 0;      // rows of the stream
    const bool rvalid = r < nx;
    const bool active = (warp & 3) * 32 < nx;  // this warp holds rows
    const int row = both ? 128 * x + r : r;    // row of the tile
    const int tok = row / G, hq = kvh * G + row - tok * G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + C::TO + x * D + lane_base;
    float m_ref = -INFINITY, l = 0.f;
    const int N = soft ? tiles_of(x) : 0;
    if (soft) {
        const bool tree = pp.parents != nullptr;
        const uint32_t *lines = reinterpret_cast<const uint32_t *>(smem + C::LINE_OFF);
        const int lim = tl.pos0 + tok;  // the token's own place
        int pos = lim;                  // and position
        if (tree) {
            int *parents = reinterpret_cast<int *>(smem + C::TREE_OFF);
            uint32_t *to = reinterpret_cast<uint32_t *>(smem + C::LINE_OFF);
            int *depth = reinterpret_cast<int *>(to + C::ROWS * kTreeWords);
            load_parents(parents, pp.parents + tl.q0, tl.i0 + tl.ntok, threadIdx.x, C::NWS * 32, first);
            named_sync(1, C::NWS * 32);
            for (int i = threadIdx.x; i < tl.ntok; i += C::NWS * 32)
                tree_line(parents, tl.i0 + i, tl.ctx, pp.window, pp.sinks, to + i * kTreeWords, depth + i);
            named_sync(1, C::NWS * 32);
            pos = tl.ctx + depth[min(tok, tl.ntok - 1)];
        }
        const int lo = pp.window > 0 ? pos - pp.window + 1 : 0;  // the row's window begins here
        const uint32_t *line = lines + min(tok, tl.ntok - 1) * kTreeWords;
        const int seen = tree ? tl.ctx : lim + 1;  // places below it are seen as far as the window lets
        // Rows are independent through both products: a warp without rows skips the tiles, and what
        // its rows of P hold reaches only its own rows of O, which are never read.
        for (int n = 0; n < (active ? N : 0); ++n) {
            const int e = 2 * x + (n & 1), j = tile_at(x, n), t = tl.place(v0 + j * BT);
            const uint32_t tS = tmem + 64 * e + lane_base;
            const bool whole = t + BT <= seen && (t >= lo || t + BT <= pp.sinks);
            const bool masked = !__all_sync(0xFFFFFFFFu, whole || !rvalid);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s_done[e], (n >> 1) & 1))) {
                misc[2] = 1;
                break;
            }
            tc_fence_after();
            float2 sv[BT / 2];
            {
                uint32_t a[32], b[32];
                tmem_ld32_issue(tS, a);
                tmem_ld32_issue(tS + 32, b);
                tmem_wait_ld();
                const float2 qs = make_float2(p.qscale, p.qscale);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    sv[k] = __fmul2_rn(make_float2(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1])), qs);
                    sv[16 + k] = __fmul2_rn(make_float2(__uint_as_float(b[2 * k]), __uint_as_float(b[2 * k + 1])), qs);
                }
            }
            if (masked) {
                uint64_t keep = low_bits(seen - t) & (~low_bits(lo - t) | low_bits(pp.sinks - t));
                if (tree && t + BT > tl.ctx) keep |= line_bits(line, t - tl.ctx);
                const uint32_t k0 = (uint32_t)keep, k1 = (uint32_t)(keep >> 32);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    if (!((k0 >> (2 * k)) & 1u)) sv[k].x = -INFINITY;
                    if (!((k0 >> (2 * k + 1)) & 1u)) sv[k].y = -INFINITY;
                    if (!((k1 >> (2 * k)) & 1u)) sv[16 + k].x = -INFINITY;
                    if (!((k1 >> (2 * k + 1)) & 1u)) sv[16 + k].y = -INFINITY;
                }
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < BT / 2; ++k) m4[k & 3] = fmaxf(m4[k & 3], fmaxf(sv[k].x, sv[k].y));
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            float alpha = 1.f;
            if (mx > m_ref) {
                if (m_ref == -INFINITY) {
                    m_ref = mx;
                } else if (mx - m_ref > 8.f) {
                    alpha = ex2(m_ref - mx);
                    m_ref = mx;
                    l *= alpha;
                }
            }
            if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) {
                // O holds the products up to the last tile's once that one is done
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&pv_done[2 * x + ((n - 1) & 1)], ((n - 1) >> 1) & 1))) {
                    misc[2] = 1;
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(tO + c, o);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t y[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(o[16 * u + k] * alpha);
                        tmem_st16(tO + c + 16 * u, y);
                    }
                }
            }
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            const float2 nm = make_float2(-mu, -mu);
            float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 v = __fadd2_rn(sv[16 * u + k], nm);
                    v.x = ex2(v.x);
                    v.y = ex2(v.y);
                    l2[k & 1] = __fadd2_rn(l2[k & 1], v);
                    y[k] = pack_bf16x2(v.x, v.y);
                }
                tmem_st16(tS + 16 * u, y);
            }
            l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
            // V rows that no row of the tile sees enter the product with weight zero, whatever they hold: those between the
            // spans, and past the end up to a multiple of 16
            const int nv = j == J - 1 ? nlast : BT;
            const int z0 = max(0, pp.sinks - t), z1 = min(BT, tl.lo - t), end = (nv + 15) & ~15;
            if (z1 > z0 || nv < end) {
                const int st = j % NS;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&v_full[st], (j / NS) & 1))) {
                    misc[2] = 1;
                    break;
                }
                const int nact = (nx + 31) / 32 * 32;  // threads of the stream's warps with rows
                for (int i = r; i < BT * C::NBLK * C::CPB; i += nact) {
                    const int k = i / (C::NBLK * C::CPB);
                    if ((k >= z0 && k < z1) || (k >= nv && k < end))
                        *reinterpret_cast<uint4 *>(ring + (st * 2 + 1) * C::TILE_BYTES +
                                                   tile_off<C>(k, i % (C::NBLK * C::CPB), 31 - __clz(p.box_rows))) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[e]);
        }
    }
    __syncthreads();
    if (soft) {
        const bool done = __all_sync(0xFFFFFFFFu, mbar_wait(&fin[0], 0) && mbar_wait(&fin[1], 0) &&
                                                         (C::NSTREAM == 1 || mbar_wait(&fin[2], 0)));
        tc_fence_after();
        const bool good = done && misc[2] == 0;
        // q and the ring are idle now: the sums leave through them, whole rows a store
        float *mine = reinterpret_cast<float *>(smem) + (x * 128 + r) * C::ROW_F;
        const float *warp_rows = mine - lane * C::ROW_F;
        const bool direct = nsplit == 1;
        const long long rq = tl.q0 + tl.i0 + tok;
        const long long prow = (rq * p.num_splits + s) * p.Hq + hq;
        const long long to = direct ? rq * p.o_sb + (long long)hq * p.o_sh : prow * D;
        const int n = min(32, nx - (r - lane));  // rows of this warp
        if (C::NSTREAM == 2 && !both) {
            // Both streams hold the same rows: each adds the other's sums to its own for half of the dims (stream 0 for
            // the first), which it gets through shared memory.
            constexpr int H = D / 2;
            const float *other = reinterpret_cast<float *>(smem) + ((1 - x) * 128 + r) * C::ROW_F;
            if (active && good) {
#pragma unroll 1
                for (int c = (1 - x) * H, i = 0; i < H / 32; ++i, c += 32) {
                    float o[32];
                    if (N > 0) tmem_ld32(tO + c, o);
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<float4 *>(mine + c + k) =
                            N > 0 ? make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                *reinterpret_cast<float2 *>(mine + D) = make_float2(m_ref, l);
            }
            named_sync(1, C::NWS * 32);
            if (active && good) {
                const float2 ml = *reinterpret_cast<const float2 *>(other + D);
                const float m = fmaxf(m_ref, ml.x), mu = m == -INFINITY ? 0.f : m;
                const float f0 = ex2(m_ref - mu), f1 = ex2(ml.x - mu), sum = l * f0 + ml.y * f1;
#pragma unroll 1
                for (int c = x * H, i = 0; i < H / 32; ++i, c += 32) {
                    float o[32];
                    if (N > 0) tmem_ld32(tO + c, o);
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(other + c + k);
                        *reinterpret_cast<float4 *>(mine + c + k) =
                            N > 0 ? make_float4(o[k] * f0 + v.x * f1, o[k + 1] * f0 + v.y * f1,
                                                o[k + 2] * f0 + v.z * f1, o[k + 3] * f0 + v.w * f1)
                                  : make_float4(v.x * f1, v.y * f1, v.z * f1, v.w * f1);
                    }
                }
                if (direct) {
                    leave<C, H, true>(warp_rows + x * H, p.out + x * H, to, sum > 0.f ? 1.f / sum : 0.f, n, lane);
                } else {
                    if (rvalid && x == 0) *reinterpret_cast<float2 *>(p.ml_part + prow * 2) = make_float2(m, sum);
                    leave<C, H, false>(warp_rows + x * H, p.o_part + x * H, to, 1.f, n, lane);
                }
            }
        } else if (active && good) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(tO + c, o);
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    *reinterpret_cast<float4 *>(mine + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            if (direct) {
                leave<C, D, true>(warp_rows, p.out, to, l > 0.f ? 1.f / l : 0.f, n, lane);
            } else {
                if (rvalid) *reinterpret_cast<float2 *>(p.ml_part + prow * 2) = make_float2(m_ref, l);
                leave<C, D, false>(warp_rows, p.o_part, to, 1.f, n, lane);
            }
        }
        if (threadIdx.x == 0 && misc[2]) {
            // a wait gave up: the copies still in flight land (bounded) before the shared memory goes
            (void)mbar_wait(q_full, 0);
            for (int i = max(0, misc[0] - NS); i < misc[0]; ++i) (void)mbar_wait(&k_full[i % NS], (i / NS) & 1);
            for (int i = max(0, misc[1] - NS); i < misc[1]; ++i)
                (void)mbar_wait(&v_full[i % NS], (i / NS) & 1);
        }
    } else if (nrows > 0 && J == 0) {  // no place at all: zero rows
        for (int i = threadIdx.x; i < nrows * (D / 8); i += C::THREADS) {
            const int ro = i / (D / 8), tk = ro / G;
            *reinterpret_cast<uint4 *>(p.out + (long long)(tl.q0 + tl.i0 + tk) * p.o_sb +
                                       (long long)(kvh * G + ro - tk * G) * p.o_sh + i % (D / 8) * 8) =
                make_uint4(0u, 0u, 0u, 0u);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                     : "memory");
    }
}

// The paged cache as [64 dims, rows, column block, kv head, page], a box of R rows of `blocks` column blocks.
bool encode_block_map(CUtensorMap *map, const void *base, int D, int Hkv, int page_size, int num_pages, int R,
                      int blocks) {
    const cuuint64_t dims[5] = {64u, (cuuint64_t)page_size, (cuuint64_t)(D / 64), (cuuint64_t)Hkv,
                                (cuuint64_t)num_pages};
    const cuuint64_t strides[4] = {(cuuint64_t)Hkv * D * 2, 128u, (cuuint64_t)D * 2,
                                   (cuuint64_t)page_size * Hkv * D * 2};
    const cuuint32_t box[5] = {64u, (cuuint32_t)R, (cuuint32_t)blocks, 1u, 1u};
    return encode_bf16(map, base, 5, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// q as [D, Hq, total_q] with its strides, a box of 64 dims x the G heads of a kv head x 128 / G tokens: 128 rows of
// 128 bytes, in the tile's row order.
bool encode_q_rows(CUtensorMap *map, const DecodeArgs &a) {
    const int G = a.Hq / a.Hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.total_q};
    // a stride over an extent of 1 is never used; give TMA a valid one
    const long long sh = a.Hq > 1 ? a.q_sh : a.D;
    const long long sb = a.total_q > 1 ? a.q_sb : (long long)a.Hq * sh;
    const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)sb * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    return encode_bf16(map, a.q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool GATHER>
dap_status launch_tc(const SpanArgs &a, cudaStream_t stream) {
    using C = SpanTcCfg<D, GATHER>;
    const int R = GATHER ? C::BT : gcd_int(a.d.page_size, C::BT), G = a.d.Hq / a.d.Hkv;
    CUtensorMap mq, mk = {}, mv = {};
    if (!encode_q_rows(&mq, a.d)) return DAP_ERR_CUDA;
    if (!GATHER &&
        (!encode_block_map(&mk, a.d.k, a.d.D, a.d.Hkv, a.d.page_size, a.d.num_pages, R, R == C::BT ? C::NBLK : 1) ||
         !encode_block_map(&mv, a.d.v, a.d.D, a.d.Hkv, a.d.page_size, a.d.num_pages, R, C::NBLK)))
        return DAP_ERR_CUDA;
    auto kern = span_tc_kernel<C>;
    static PerDeviceOcc occ = {};
    if (prepare_kernel(kern, C::THREADS, C::SMEM, &occ, 100) <= 0) return DAP_ERR_CUDA;
    const long long grid = (long long)a.d.num_tiles * a.d.Hkv * a.d.num_splits;
    if (grid > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    const SpanParams p = span_params(a, R);
    if (launch_dependent_smem(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, mq, mk, mv, p, G) !=
        cudaSuccess)
        return DAP_ERR_CUDA;
    return launch_span_combine<D>(a, p, C::ROWS / G, stream);
}

template <bool GATHER>
dap_status tc_dims(const SpanArgs &a, cudaStream_t stream) {
    switch (a.d.D) {
        case 64: return launch_tc<64, GATHER>(a, stream);
        case 128: return launch_tc<128, GATHER>(a, stream);
        case 256: return launch_tc<256, GATHER>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

}  // namespace

dap_status launch_span_tc(const SpanArgs &a, cudaStream_t stream) {
    return a.d.page_size % 8 != 0 ? tc_dims<true>(a, stream) : tc_dims<false>(a, stream);
}

bool read_errors_span_tc(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
