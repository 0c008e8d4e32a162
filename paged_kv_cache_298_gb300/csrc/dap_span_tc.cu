// dap_span_tc.cu -- attention over spans of the paged cache (dap_span.cuh has the operation) for many query rows, on the
// tcgen05 tensor cores: verification of larger trees, chunks of prompts behind a window.
//
// One CTA takes a work tile of query rows of one kv head (row r: new token r / G of the tile, head r % G) against one chunk of
// the tile's spans, in streams of 128 rows: one stream, in which case two CTAs share an SM (one at D = 256), or two (WIDE),
// which share every K/V tile (span_tokens_per_tile has the rule).
//   shared memory: q (128-byte swizzled, one TMA copy per 64 dims of 128 rows), a ring of K/V tiles of 64 keys.  K tiles are
//                  column block major, [D / 64][64 keys][128 bytes], a copy per page run and column block; V tiles one box per
//                  page run, [D / 64][R keys][128 bytes], since a product takes 16 keys of V at a time (row gather: both
//                  column block major);
//   tensor memory (lane = row): S  columns [128 x + 64 e, + 64) of stream x: fp32 scores of tile n in buffer e = n & 1; P (bf16
//                  pairs) overwrites the first 32 once they are read;  O  columns [TO + x D, + D): fp32 accumulator.
// Warps: four softmax warps a stream (thread = row), a producer each for K and V, one a stream that issues its scores, one
// that issues the products with V.  S(n + 2) needs only PV(n), whose P it replaces.
//   * Spans: a tile has to be masked by row where an end of a window, the new tokens or a tree's nodes lie in it.  A row's
//     mask of the 64 keys is one 64-bit word, made of its bounds and its line of ancestors; tiles that every row of a warp
//     sees whole, nearly all, skip it.
//   * V rows that no row of the tile sees are zeroed by the softmax threads, before they hand over the tile's weights.
//   * With one split the rows leave as bf16 outputs, whole rows a store, and no combine follows.
// Bound, at many rows: the chain of a tile, 1750 cycles for 256 rows x 64 keys (D = 128), of which the products take 1330 - 1580
// (24 of them, 50 to 66 cycles each whatever their size) and a softmax warp 930 - 1070; a CTA's start and end, 15,000 cycles,
// most of it waits for memory, are what a second CTA on the SM covers.  Measured and not kept: score products of 128 keys with
// one buffer a stream (1.28 us a 64-key tile of 256 rows for 0.91: the chain S, softmax, PV is then in line), weights taken
// against the old reference while the maximum is found (0.96 - 1.0), one producer warp for K and V (0.96).
// Softmax: base 2, scores rounded once; the running maximum is moved lazily (O and l are rescaled only when a tile's maximum
// passes the reference by more than 2^8), so the weights stay <= 256.  They are rounded to bf16 for the product with V, whose
// type is bf16; l sums them in fp32 before that rounding.  Summing the rounded ones brings the error against 64 bits from 0.0023 of
// the output to 0.0022 (0.0017 of it is the output's own rounding) and costs 3 to 5%, since the softmax warps' chain is what
// bounds a tile: 163 us for 157 on 64 trees of 64 nodes, 152.5 for 145 on four chunks of 1021 tokens.
#include <algorithm>

#include "dap_span.cuh"
#include "dap_tc.cuh"

namespace dap {

namespace {

// PAIR: 128 rows in one stream, two CTAs an SM; WIDE: 256 rows in two streams, one CTA an SM; DEEP: 128 rows and one CTA an SM
// with all of its memory for the ring (D = 256: always).
enum Shape { PAIR, WIDE, DEEP };
template <int D_, Shape SHAPE, bool GATHER_>
struct SpanTcCfg {
    static constexpr bool GATHER = GATHER_, SWZ = true;
    static constexpr int D = D_, BT = 64;
    static constexpr int ROWB = D * 2, SWB = 128, NBLK = ROWB / SWB, CPB = SWB / 16;
    static constexpr int TILE_BYTES = BT * ROWB;  // K or V of one tile
    static constexpr int NSTREAM = SHAPE == WIDE ? 2 : 1, ROWS = 128 * NSTREAM, MINB = SHAPE == PAIR ? 2 : 1;
    // K/V tiles in the ring
    static constexpr int NS = D == 256 ? 2 : SHAPE == PAIR ? (D == 64 ? 4 : 2) : SHAPE == WIDE ? (D == 64 ? 6 : 4) : (D == 64 ? 10 : 5);
    static constexpr int NWS = 4 * NSTREAM, PRODUCER = NWS, ISSUER = NWS + 2, PV = ISSUER + NSTREAM,
                         THREADS = (PV + 1) * 32;
    static constexpr int TO = SHAPE == WIDE || D == 256 ? 256 : 128, TMEM_COLS = 2 * TO;
    static constexpr int QBLK = 128 * 128, Q_BYTES = NSTREAM * NBLK * QBLK;  // 64 dims of 128 rows; all of q
    static constexpr int RING_OFF = Q_BYTES, BAR_OFF = RING_OFF + NS * 2 * TILE_BYTES;
    // barriers: k_full, k_empty, v_full, v_empty [NS], s_done, p_ready, pv_done [stream][buffer], q_full, fin[3]
    static constexpr int NBAR = 4 * NS + 16;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    // a tree's parents, lines and depths (G = 1: as many tokens as rows)
    static constexpr int TREE_OFF = MISC_OFF + 32, LINE_OFF = TREE_OFF + kTreeMost * 4;
    static constexpr int SMEM = LINE_OFF + ROWS * (kTreeWords + 1) * 4 + 1024;  // + slack to align the base
    static constexpr int ROW_B = D * 4 + 16;  // bytes of a row of sums on its way out (the 16: no bank conflicts)
    static_assert(SHAPE == DEEP || D <= 128, "tensor memory");
    static_assert(TO + NSTREAM * D <= TMEM_COLS && 128 * NSTREAM <= TO, "tensor memory");
    static_assert(SMEM <= 227 * 1024 / MINB, "shared memory");
    static_assert(MINB == 2 || SMEM > 114 * 1024, "one CTA an SM: a second would wait for tensor memory");
    static_assert(ROWS * ROW_B <= BAR_OFF, "the sums on their way out fit the place of q and the ring");
    // (a stream's rows leave when its own products are done; all scores are, but not the other stream's last product with V)
    static_assert(NSTREAM == 1 || 128 * ROW_B <= RING_OFF + TILE_BYTES, "the first stream's rows end before the first V tile");
};

// 32 columns of a row's sums in shared memory, as fp32 or, with BF16, times `f` and rounded (rows are ROW_B bytes apart).
template <bool BF16>
__device__ __forceinline__ void put32(uint8_t *row, int c, const float (&o)[32], float f) {
    if constexpr (BF16) {
#pragma unroll
        for (int k = 0; k < 32; k += 8)
            *reinterpret_cast<uint4 *>(row + (c + k) * 2) =
                make_uint4(pack_bf16x2(o[k] * f, o[k + 1] * f), pack_bf16x2(o[k + 2] * f, o[k + 3] * f),
                           pack_bf16x2(o[k + 4] * f, o[k + 5] * f), pack_bf16x2(o[k + 6] * f, o[k + 7] * f));
    } else {
#pragma unroll
        for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4 *>(row + (c + k) * 4) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
    }
}

// `n` rows that a warp has in shared memory to global memory, BYTES of each: row i of the tile's rows first, first + 1, ..
// is (token i / G, head i % G) and goes to out + token * st + head * sh.  Whole rows a store, eight loads ahead.
template <int BYTES, int ROW_B>
__device__ __forceinline__ void leave(const uint8_t *rows, uint8_t *out, int first, int n, int G, long long st, long long sh,
                                      int lane) {
    constexpr int W = BYTES < 512 ? BYTES : 512, LPR = W / 16, RPI = 32 / LPR, U = 32 / RPI < 8 ? 32 / RPI : 8;
    static_assert(BYTES % W == 0, "whole rows");
    __syncwarp();
    const int sub = lane / LPR, gs = 31 - __clz(G);
#pragma unroll
    for (int c0 = 0; c0 < BYTES; c0 += W) {
        const int c = c0 + lane % LPR * 16;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += RPI * U) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const uint4 *>(rows + (i0 + u * RPI + sub) * ROW_B + c);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * RPI + sub;
                if (i < n)
                    *reinterpret_cast<uint4 *>(out + ((first + i) >> gs) * st + ((first + i) & (G - 1)) * sh + c) = v[u];
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
__global__ void __launch_bounds__(C::THREADS, C::MINB)
    span_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, const SpanParams pp, const int G,
                   const bool longest_first) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = aligned_smem<C>(smem_raw);
    constexpr int BT = C::BT, NS = C::NS, D = C::D;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
    uint64_t *s_done = v_empty + NS, *p_ready = s_done + 4, *pv_done = p_ready + 4;  // [2 stream + buffer]
    uint64_t *q_full = pv_done + 4, *fin = q_full + 1;
    // [0], [1] K and V tiles issued, [2] abort, [3] the work tile, [4] tensor memory
    volatile int *misc = reinterpret_cast<volatile int *>(smem + C::MISC_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF) + 4;
    uint8_t *ring = smem + C::RING_OFF;

    const int units = p.num_tiles * p.Hkv;
    const int s = (int)(blockIdx.x / units);
    const int rem = (int)(blockIdx.x - s * units);
    const int slot = rem / p.Hkv;
    const int kvh = rem - slot * p.Hkv;

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

    const int qt = C::ROWS / G;
    const bool first = s == 0 && kvh == 0;
    auto tile_of = [&](int i, bool report, SpanTile *t) -> bool {
        const int wb = p.tile_batch[i], bb = (wb >= 0 && wb < p.B) ? wb : 0;
        return span_tile(pp, wb, p.tile_index[i], p.qo_indptr[bb], p.qo_indptr[bb + 1], p.seq_lens[bb], qt, report, t);
    };
    int w = slot;
    if (longest_first) {
        // CTAs start in the order of their numbers, so the slot-th longest tile goes to this one: every CTA ranks all tiles.
        int *len = reinterpret_cast<int *>(ring);
        SpanTile t;
        for (int i = threadIdx.x; i < p.num_tiles; i += C::THREADS) len[i] = tile_of(i, false, &t) ? t.len : -1;
        __syncthreads();
        for (int i = warp; i < p.num_tiles; i += C::THREADS / 32) {
            const int mine = len[i];
            int rank = 0;
            for (int k = lane; k - lane < p.num_tiles; k += 32)
                rank += __popc(__ballot_sync(0xFFFFFFFFu, k < p.num_tiles && (len[k] > mine || (len[k] == mine && k < i))));
            if (rank == slot && lane == 0) misc[3] = i;
        }
        fence_async_smem();  // (the ring's copies come after these reads and writes)
        __syncthreads();
        w = misc[3];
    }
    SpanTile tl;
    const bool live = tile_of(w, threadIdx.x == 0 && first, &tl);
    const int nsplit = live ? span_splits(tl, p.chunk) : 0;
    const int nrows = s < nsplit ? tl.ntok * G : 0;
    const int v0 = s * p.chunk, v1 = s < nsplit ? min(tl.len, v0 + p.chunk) : v0;
    const int J = max(0, v1 - v0 + BT - 1) / BT;  // K/V tiles of this CTA
    const bool work = nrows > 0 && J > 0;
    const int streams = C::NSTREAM == 2 && nrows > 128 ? 2 : 1;  // that have rows
    auto rows_of = [&](int x) { return max(0, min(128, nrows - 128 * x)); };
    if (threadIdx.x < C::NBAR) {  // a thread a barrier
        const int i = threadIdx.x, e = i - 4 * NS;
        uint32_t n = 1;  // s_done, pv_done, fin: a commit; q_full: bytes
        if (i < NS || (i >= 2 * NS && i < 3 * NS)) n = full_arrivals<C>();  // k_full, v_full
        else if (i < 2 * NS) n = streams;  // k_empty: a commit of every stream's scores (v_empty: one, the last product's)
        else if (e >= 4 && e < 8) n = (uint32_t)max(1, (rows_of((e - 4) >> 1) + 31) / 32);  // p_ready: the warps with rows
        mbar_init(k_full + i, n);
        fence_barrier_init();
    }
    if (threadIdx.x < 3) misc[threadIdx.x] = 0;
    // The producers ask for their first page ids meanwhile (32 entries of the first span each, and of the window).
    const int32_t *table = p.block_table + (long long)(work ? tl.b : 0) * p.max_pages;
    const bool jumps = work && tl.gap > 0 && v0 < tl.sink_end && tl.sink_end < v1;
    const int e_first = work ? tl.place(v0) / p.page_size : 0, e_jump = jumps ? tl.place(tl.sink_end) / p.page_size : e_first;
    const bool asks = !C::GATHER && work && (warp == C::PRODUCER || warp == C::PRODUCER + 1);
    PageWindow pages(table, e_first, asks ? p.max_pages : 0, lane), beyond(table, e_jump, asks && jumps ? p.max_pages : 0, lane);
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
        const int R = p.box_rows;
        uint64_t *full = tensor ? v_full : k_full, *empty = tensor ? v_empty : k_empty;
        uint8_t *place = ring + tensor * C::TILE_BYTES;
        int done = 0;  // tiles issued
        auto load_q = [&] {  // 64 dims of 128 rows a copy (rows past the tile's tokens are never read)
            if (tensor == 1 && lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)(streams * C::NBLK * C::QBLK));
                for (int x = 0; x < streams; ++x)
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
                        next.pg[k] = table[(hidden(t, 1) ? tl.lo : t) / p.page_size];
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
            load_q();
            for (; done < J; ++done) {
                const int st = done % NS, v = v0 + done * BT, t = tl.place(v);
                if (jumps && v == tl.sink_end) {
                    start(t);
                    pages = beyond;
                }
                const int nbox = (min(BT, v1 - v) + R - 1) / R;
                int pg = pages.at(e, e0);
                const bool has = j < nbox && !hidden(t + j * R, R);
                const int copied = __popc(__ballot_sync(0xFFFFFFFFu, has)) / kb;
                if (done >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((done / NS) - 1) & 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(copied * R * C::ROWB));
                __syncwarp();
                if (has) {
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
        const int Ju = same(J), last = same(nlast), live_streams = same(streams);
        const uint32_t tm = same(tmem);
        const uint32_t sQ = smem_addr(smem), sR = smem_addr(ring);
        auto wait = [&](uint64_t *b0, int n0, uint64_t *b1, int n1) -> bool {
            const bool odd = lane & 1;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(odd ? b1 : b0, (odd ? n1 : n0) & 1)) != 0;
            if (C::GATHER) fence_async_smem();  // (K and V rows were copied by the generic proxy)
            tc_fence_after();
            return ok;
        };
        bool ok = true;
        if (role < C::NSTREAM) {  // S(n), once PV(n - 2), whose P it replaces, is done
            const uint64_t dQ = sw128_desc(sQ + role * C::NBLK * C::QBLK, 16, 1024);
            for (int n = 0; n < (role < live_streams ? Ju : 0); ++n) {
                const int st = n % NS, e = 2 * role + (n & 1);
                if (!(ok = n >= 2 ? wait(&k_full[st], n / NS, &pv_done[e], (n - 2) >> 1) : wait(&k_full[st], n / NS, q_full, 0)))
                    break;
                const uint64_t dK = sw128_desc(sR + st * 2 * C::TILE_BYTES, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_bf16(tm + 64 * e, dQ + (((i >> 2) * C::QBLK + (i & 3) * 32) >> 4),
                                  dK + (((i >> 2) * CS + (i & 3) * 32) >> 4), idS, i > 0);
                    umma_commit(&s_done[e]);
                    umma_commit(&k_empty[st]);
                }
                __syncwarp();
            }
        } else {  // O += P(n) . V(n), stream by stream
            // A V tile is made of boxes [column block][vR keys][128 bytes]; byte offset of key 16 i and the strides of
            // the product's blocks of 64 dims and groups of 8 keys.
            const int vR = same(p.box_rows);
            const uint32_t v_lbo = vR * 128, v_sbo = vR == 8 ? 8 * C::ROWB : 1024;
            auto v_off = [&](int i) -> uint32_t { return (i * 16 / vR * vR * C::ROWB + i * 16 % vR * 128) >> 4; };
            const uint32_t a1 = v_off(1), a2 = v_off(2), a3 = v_off(3);
            for (int n = 0; ok && n < Ju; ++n) {
                const int st = n % NS, nv = n == Ju - 1 ? last : BT;
                const uint64_t dV = sw128_desc(sR + (st * 2 + 1) * C::TILE_BYTES, v_lbo, v_sbo);
                for (int x = 0; x < live_streams; ++x) {
                    const int e = 2 * x + (n & 1);
                    if (!(ok = wait(&p_ready[e], n >> 1, &v_full[st], n / NS))) break;
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < BT / 16; ++i)
                            if (i * 16 < nv)
                                umma_bf16_tmem_a(tm + C::TO + x * D, tm + 64 * e + i * 8,
                                                 dV + (i == 0 ? 0u : i == 1 ? a1 : i == 2 ? a2 : a3), idO, n > 0 || i > 0);
                        umma_commit(&pv_done[e]);
                        if (x == live_streams - 1) umma_commit(&v_empty[st]);  // (a commit covers all products before it)
                    }
                    __syncwarp();
                }
            }
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
    const int row = 128 * x + r;               // row of the tile
    const int tok = row / G, hq = kvh * G + row - tok * G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + C::TO + x * D + lane_base;
    float m_ref = -INFINITY, l = 0.f;
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
        for (int n = 0; n < (active ? J : 0); ++n) {
            const int e = 2 * x + (n & 1), t = tl.place(v0 + n * BT);
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
            const int nv = n == J - 1 ? nlast : BT;
            const int z0 = max(0, pp.sinks - t), z1 = min(BT, tl.lo - t), end = (nv + 15) & ~15;
            if (z1 > z0 || nv < end) {
                const int st = n % NS;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&v_full[st], (n / NS) & 1))) {
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
        // (with a wait that gave up, misc[2] was set before the barrier above)
        const bool good = misc[2] == 0 &&
                          (!active || __all_sync(0xFFFFFFFFu, mbar_wait(&pv_done[2 * x + ((J - 1) & 1)], ((J - 1) >> 1) & 1)));
        tc_fence_after();
        if (active && good) {
            // q and the ring are idle now: the sums leave through them
            uint8_t *mine = smem + row * C::ROW_B;
            const uint8_t *warp_rows = mine - lane * C::ROW_B;
            const bool direct = nsplit == 1;
            const int n = min(32, nx - (r - lane));  // rows of this warp
            const long long t0 = tl.q0 + tl.i0;
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(tO + c, o);
                if (direct) put32<true>(mine, c, o, inv);
                else put32<false>(mine, c, o, 1.f);
            }
            if (direct) {
                leave<D * 2, C::ROW_B>(warp_rows,
                                       reinterpret_cast<uint8_t *>(p.out + t0 * p.o_sb + (long long)kvh * G * p.o_sh),
                                       row - lane, n, G, p.o_sb * 2, p.o_sh * 2, lane);
            } else {
                const long long prow = (t0 * p.num_splits + s) * p.Hq + kvh * G;
                if (rvalid)
                    *reinterpret_cast<float2 *>(p.ml_part + (((t0 + tok) * p.num_splits + s) * p.Hq + hq) * 2) =
                        make_float2(m_ref, l);
                leave<D * 4, C::ROW_B>(warp_rows, reinterpret_cast<uint8_t *>(p.o_part + prow * D), row - lane, n, G,
                                       (long long)p.num_splits * p.Hq * D * 4, D * 4, lane);
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
    if (work && warp == 0) (void)mbar_wait(&fin[lane <= C::NSTREAM ? lane : 0], 0);  // all products are done
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

template <int D, Shape SHAPE, bool GATHER>
dap_status launch_tc(const SpanArgs &a, cudaStream_t stream) {
    using C = SpanTcCfg<D, SHAPE, GATHER>;
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
    const SpanParams p = span_params(a, R, C::BT);
    // More CTAs than fit at once, of unequal lengths (a window makes them about equal), and not so many that ranking them
    // takes longer than the end of the last ones would: 64 trees of 64 nodes behind 256 .. 4096 keys, 154 us for 170.
    const bool longest_first = a.window == 0 && grid > (long long)C::MINB * dap_device_sm_count() && a.d.num_tiles > 1 &&
                               a.d.num_tiles <= 128;
    if (launch_dependent_smem(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, mq, mk, mv, p, G,
                              longest_first) != cudaSuccess)
        return DAP_ERR_CUDA;
    return launch_span_combine<D>(a, p, C::ROWS / G, stream);
}

// DEEP where every CTA has an SM to itself (16 trees of 16 nodes behind 2048 keys, 128 CTAs: 29.9 us for 35.6).
template <int D, bool GATHER>
dap_status tc_shape(const SpanArgs &a, cudaStream_t stream) {
    if (a.d.tokens_per_tile * (a.d.Hq / a.d.Hkv) == 256) return launch_tc<D, WIDE, GATHER>(a, stream);
    if ((long long)a.d.num_tiles * a.d.Hkv * a.d.num_splits <= dap_device_sm_count()) return launch_tc<D, DEEP, GATHER>(a, stream);
    return launch_tc<D, PAIR, GATHER>(a, stream);
}

template <bool GATHER>
dap_status tc_dims(const SpanArgs &a, cudaStream_t stream) {
    switch (a.d.D) {
        case 64: return tc_shape<64, GATHER>(a, stream);
        case 128: return tc_shape<128, GATHER>(a, stream);
        case 256: return launch_tc<256, DEEP, GATHER>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

}  // namespace

dap_status launch_span_tc(const SpanArgs &a, cudaStream_t stream) {
    return a.d.page_size % 8 != 0 ? tc_dims<true>(a, stream) : tc_dims<false>(a, stream);
}

bool read_errors_span_tc(unsigned int *flags, bool clear) { return read_span_errors(flags, clear); }

}  // namespace dap
