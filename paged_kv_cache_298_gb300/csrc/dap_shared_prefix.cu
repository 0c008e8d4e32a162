// dap_shared_prefix.cu -- the prefix part of the shared-prefix decode on the tcgen05 tensor cores, and
// the combine that merges prefix and suffix partials (dap_shared.cuh has the operation).
//
// One CTA takes a tile of up to 256 query rows of one kv head (row r: sequence r / G of the tile, head
// r % G), or 128 at D = 256, against one chunk of the group's prefix.  Two streams of 128 rows (one at
// D = 256) keep the tensor cores busy: stream x has rows [128 x, 128 x + 128) of the tile and every K/V
// tile; with at most 128 rows both streams hold the same rows and take every other K/V tile, merged through
// shared memory at the end.
//   shared memory: q (128-byte swizzled, one TMA copy per 64 dims of 128 rows), a ring of K/V tiles of 64
//                  keys.  K tiles are column block major, [D / 64][64 keys][128 bytes], as the product with
//                  N = 64 keys wants its 8-key groups one stride apart: a copy per page run and column block (one in
//                  all for page sizes that are multiples of 64).  V tiles are made of one box per page run,
//                  [D / 64][R keys][128 bytes], since a product takes 16 keys of V at a time: half the copies.
//                  Row gather: both column block major;
//   tensor memory (lane = row): S  columns [128 x + 64 e, + 64)  fp32 scores of tile n in buffer e = n & 1;
//                                  P (bf16 pairs) overwrites the first 32 once they are read;
//                               O  columns [256 + x D, + D)  fp32 accumulator.
// Warps: four softmax warps a stream (thread = row), a producer each for K and V, one a stream that issues its
// scores and one that issues all products with V.  S(n + 2) needs only PV(n), whose P it replaces, so the scores
// are there when the softmax gets to them.
// Bound: the products, in this shape.  At D = 128 those of a 64-key tile of 256 rows take 1344 cycles (a microbenchmark:
// 50 an S product, N = 64, whose operands both come from shared memory, 66 a PV product, N = 128); at the PV products'
// rate the same work is 1024.  A tile takes 0.82 us (10 TFLOP/s an SM), with at most 128 rows 0.43 us at page sizes
// that are multiples of 64 and 0.65 at 16, where the producers' copies bound it; 0.86 us at D = 256 (128 rows; 1.00 at
// page size 16).
// Why these warps (cycles of a tile at the time, D = 128): one score buffer a stream, every step of the chain S,
// softmax, PV waiting for the last: 3130; two buffers, one issuing warp a stream: 2100, as PV(n) has to end before
// the same warp can go on to S(n + 2); one warp for everything, PV_0(n), S_1(n + 1), PV_1(n), S_0(n + 2): 2770, as
// a wait on a barrier takes 60 cycles even when it is complete and a commit 55, all of them in line; one warp for the
// scores of both: 1990; one producer warp for K and V: 1800, and 0.72 us a tile whatever its rows.
// L2 prefetch of later tiles, by TMA or by loads, measured slower (prefix alone 71 against 90 us): it takes the
// producers' time, and the ring already covers the latency.
// Softmax: base 2, scores rounded once; the running maximum is moved lazily (O and l are rescaled only
// when a tile's maximum passes the reference by more than 2^8), so the weights stay <= 256.  The
// weights are rounded to bf16 for the product with V, whose type is bf16; l sums them in fp32, before that
// rounding (the suffix kernel's l, whose weights are at hand as bf16 fragments, after it: either is within 2^-8 of the other).
#include "dap_shared.cuh"
#include "dap_tc.cuh"

namespace dap {

namespace {

template <int D_, bool GATHER_>
struct PrefixCfg {
    static constexpr bool GATHER = GATHER_, SWZ = true;
    static constexpr int D = D_, BT = 64;
    static constexpr int ROWB = D * 2, SWB = 128, NBLK = ROWB / SWB, CPB = SWB / 16;
    static constexpr int TILE_BYTES = BT * ROWB;              // K or V of one tile
    static constexpr int NSTREAM = D == 256 ? 1 : 2;
    static constexpr int NS = D == 64 ? 6 : D == 128 ? 4 : 2;  // K/V tiles in the ring
    static constexpr int NWS = 4 * NSTREAM, PRODUCER = NWS, ISSUER = NWS + 2, PV = ISSUER + NSTREAM,
                         THREADS = (PV + 1) * 32;
    static constexpr int TO = 256, TMEM_COLS = 512;
    static constexpr int QBLK = 128 * 128, Q_BYTES = NSTREAM * NBLK * QBLK;  // 64 dims of 128 rows; all of q
    static constexpr int RING_OFF = Q_BYTES, BAR_OFF = RING_OFF + NS * 2 * TILE_BYTES;
    // barriers: k_full, k_empty, v_full, v_empty [NS], s_done, p_ready, pv_done [stream][buffer], q_full, fin[3], tail
    static constexpr int NBAR = 4 * NS + 17;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr int USED = MISC_OFF + 32 + 1024;  // + slack to align the base to 1024
    // More than half an SM's shared memory, so that two prefix CTAs never share an SM (the second would wait for
    // tensor memory).  A ring small enough for a suffix CTA beside it (three tiles at D = 128) measured slower: the
    // two slow each other down by more than the suffix CTA gets done.
    static constexpr int SMEM = USED;
    static constexpr int ROW_F = D + 4;  // floats of a row of sums on its way out (the 4: no bank conflicts)
    static_assert(SMEM > 114 * 1024 && SMEM <= 227 * 1024, "shared memory");
    static_assert(NSTREAM * 128 * ROW_F * 4 <= BAR_OFF, "the sums on their way out fit the place of q and the ring");
};

// `n` rows of sums (NC of their floats) that a warp has in shared memory, ROW_F apart, to their places (element `to` of
// `out` for the lane's row): whole rows a store, eight stores' loads ahead of the first.
template <class C, int NC>
__device__ __forceinline__ void store_rows(const float *rows, float *out, long long to, int n, int lane) {
    constexpr int W = NC < 128 ? NC : 128, LPR = W / 4, RPI = 32 / LPR, U = 8;
    static_assert(NC % W == 0 && 32 % (RPI * U) == 0, "whole batches");
    __syncwarp();
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += W) {
        const int c = c0 + lane % LPR * 4;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += RPI * U) {
            float4 v[U];
            long long at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * RPI + lane / LPR;
                at[u] = __shfl_sync(0xFFFFFFFFu, to, i);
                v[u] = *reinterpret_cast<const float4 *>(rows + i * C::ROW_F + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * RPI + lane / LPR < n) *reinterpret_cast<float4 *>(out + at[u] + c) = v[u];
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV, const SharedParams pp, const int G) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = aligned_smem<C>(smem_raw);
    constexpr int BT = C::BT, NS = C::NS, D = C::D;
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
    uint64_t *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
    uint64_t *s_done = v_empty + NS, *p_ready = s_done + 4, *pv_done = p_ready + 4;  // [2 stream + buffer]
    uint64_t *q_full = pv_done + 4, *fin = q_full + 1, *tail = fin + 3;
    // [0], [1] K and V tiles issued, [2] abort, [4] tensor memory
    volatile int *misc = reinterpret_cast<volatile int *>(smem + C::MISC_OFF);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF) + 4;
    uint8_t *ring = smem + C::RING_OFF;

    const int units = pp.num_tiles * p.Hkv;
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
    // Nothing global is read before the wait; the suffix kernel may start after it, and once every CTA holds its tensor
    // memory: a kernel further down the stream may take some before its own wait, and a CTA that still waited for columns
    // held by a kernel that waits for this one would never get them.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // (group, first sequence of the group, first sequence of the tile, sequences)
    const int4 tl = __ldg(reinterpret_cast<const int4 *>(pp.tiles) + w);
    const bool valid = tl.x >= 0 && tl.x < pp.num_groups && tl.y >= 0 && tl.y < p.B && tl.z >= 0 && tl.w >= 1 &&
                       tl.w <= pp.seqs_per_tile && tl.w <= p.B - tl.z;
    const int q0 = tl.y, first = tl.z, nseq = valid ? tl.w : 0;
    const int P = valid ? group_prefix(pp, tl.x) : 0;
    if (!valid && threadIdx.x == 0 && s == 0 && kvh == 0) flag_error(DAP_DEVERR_QMAP);
    const int nrows = nseq * G;
    const int tok0 = min(P, s * pp.prefix_chunk), tok1 = min(P, tok0 + pp.prefix_chunk);
    const int J = (tok1 - tok0 + BT - 1) / BT;  // K/V tiles of this CTA
    const bool work = nrows > 0 && J > 0;
    const bool both = C::NSTREAM == 2 && nrows > 128;   // the streams have rows of their own
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
        mbar_init(tail, 1);
        misc[0] = misc[1] = misc[2] = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();  // barriers and the tensor-memory address are visible
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t CS = BT * 128;  // bytes between column blocks of a tile
    constexpr uint32_t idS = idesc_bf16(128, BT, 0), idO = idesc_bf16(128, D, 1);
    const int nlast = tok1 - (tok0 + (J - 1) * BT);  // keys of the last tile
    const bool ragged = work && nlast % 16 != 0;     // its V rows up to a multiple of 16 are zeroed

    if (work && (warp == C::PRODUCER || warp == C::PRODUCER + 1)) {
        // A producer warp each for K and V: a tile's chain of barrier, page and copy takes a warp some 700 cycles a
        // tensor, whatever the size of the copies.
        const int tensor = warp - C::PRODUCER;
        const int32_t *table = p.block_table + (long long)q0 * p.max_pages;
        const int R = p.box_rows;
        uint64_t *full = tensor ? v_full : k_full, *empty = tensor ? v_empty : k_empty;
        uint8_t *place = ring + tensor * C::TILE_BYTES;
        int done = 0;  // tiles issued
        auto load_q = [&] {  // 64 dims of 128 rows a copy (rows past the tile's end are never read)
            if (tensor == 0 && lane == 0) {
                const int parts = both ? 2 : 1;
                mbar_arrive_expect_tx(q_full, (uint32_t)(parts * C::NBLK * C::QBLK));
                for (int x = 0; x < parts; ++x)
                    for (int cb = 0; cb < C::NBLK; ++cb)
                        tma_load_3d(smem + (x * C::NBLK + cb) * C::QBLK, &mapQ, cb * 64, kvh * G, first + x * (128 / G),
                                    q_full);
            }
            __syncwarp();
        };
        if constexpr (C::GATHER) {
            RowWalk<C> walk(table, tok0, p, lane);
            load_q();
            for (; done < J; ++done) {
                const int st = done % NS, t = tok0 + done * BT;
                RowPages<C> rp;
                walk.next(rp);
                if (done >= NS && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], ((done / NS) - 1) & 1))) break;
                gather_rows<C, false>(place + st * 2 * C::TILE_BYTES, tensor ? p.v_cache : p.k_cache, nullptr, rp,
                                      min(BT, tok1 - t), kvh, p, &full[st], lane);
            }
        } else {
            // K: lane = (box j, column block cb), or a whole tile where a page has one; V: lane = box, all blocks.  A
            // lane steps the entry and the row of its box from tile to tile (no division).
            const CUtensorMap *map = tensor ? &mapV : &mapK;
            const int kb = tensor || R == BT ? 1 : C::NBLK;
            const int j = lane / kb, cb = lane % kb;
            const int to = tensor ? j * R * C::ROWB : cb * (int)CS + j * R * 128;
            int e0 = tok0 / p.page_size, row0 = tok0 - e0 * p.page_size;
            PageWindow pages(table, e0, p.max_pages, lane);
            load_q();
            const int dq = BT / p.page_size, dr = BT - dq * p.page_size;
            int e = e0, row = row0 + (j * R < BT ? j * R : 0);  // (lanes without a box follow the tile's first)
            for (; row >= p.page_size; ++e) row -= p.page_size;
            for (; done < J; ++done) {
                const int st = done % NS;
                const int nbox = (min(BT, tok1 - (tok0 + done * BT)) + R - 1) / R;
                int pg = pages.at(e, e0);
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
                e += dq;
                if ((row += dr) >= p.page_size) {
                    row -= p.page_size;
                    ++e;
                }
                e0 += dq;
                if ((row0 += dr) >= p.page_size) {
                    row0 -= p.page_size;
                    ++e0;
                }
            }
        }
        if (done < J) misc[2] = 1;
        if (lane == 0) misc[tensor] = done;
        __syncwarp();
        if (tensor == 1 && ragged && done == J) {
            // V rows past the end enter the last product with weight zero, whatever the page holds
            const int st = (J - 1) % NS;
            if (__all_sync(0xFFFFFFFFu, mbar_wait(&v_full[st], ((J - 1) / NS) & 1))) {
                const int nz = 16 - nlast % 16;
                for (int e = lane; e < nz * C::NBLK * C::CPB; e += 32)
                    *reinterpret_cast<uint4 *>(ring + (st * 2 + 1) * C::TILE_BYTES +
                                               tile_off<C>(nlast + e / (C::NBLK * C::CPB), e % (C::NBLK * C::CPB),
                                                           31 - __clz(R))) =
                        make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(tail);
            } else {
                misc[2] = 1;
            }
        }
        // every commit on these barriers has arrived before the CTA ends
        for (int i = max(0, J - NS); i < J && done == J; ++i)
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[i % NS], (i / NS) & 1))) {
                misc[2] = 1;
                break;
            }
    } else if (work && warp >= C::ISSUER) {
        // The whole warp runs its loop with values that are the same in every lane (and known to be), one lane
        // issues: descriptors then stay in uniform registers.  Two barriers are polled at a time, each by half the
        // lanes.
        auto same = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
        const int role = same(warp - C::ISSUER);  // a stream's scores; NSTREAM: all products with V
        const int Ju = same(J), last = same(nlast);
        const bool two = same(both) != 0, tailed = same(ragged) != 0;
        const uint32_t tm = same(tmem);
        const int step = two || C::NSTREAM == 1 ? 1 : 2;  // tile n of stream x is step * n + (step == 2 ? x : 0)
        const uint32_t sQ = smem_addr(smem), sR = smem_addr(ring);
        // A V tile is made of boxes [column block][vR keys][128 bytes]; byte offset of key 16 i and the strides of
        // the product's blocks of 64 dims and groups of 8 keys.
        const int vR = same(p.box_rows);
        const uint32_t v_lbo = vR * 128, v_sbo = vR == 8 ? 8 * C::ROWB : 1024;
        auto v_off = [&](int i) -> uint32_t { return i * 16 / vR * vR * C::ROWB + i * 16 % vR * 128; };
        const uint32_t v1 = v_off(1) >> 4, v2 = v_off(2) >> 4, v3 = v_off(3) >> 4;
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
            const bool end = j == Ju - 1;
            if (!(end && tailed ? wait(&p_ready[e], n >> 1, tail, 0) : wait(&p_ready[e], n >> 1, &v_full[st], j / NS)))
                return false;
            const int nv = end ? last : BT;
            const uint64_t dV = sw128_desc(sR + (st * 2 + 1) * C::TILE_BYTES, v_lbo, v_sbo);
            const uint32_t tP = tm + 64 * e, tOx = tm + C::TO + x * D;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < BT / 16; ++i)
                    if (i * 16 < nv)
                        umma_bf16_tmem_a(tOx, tP + i * 8, dV + (i == 0 ? 0u : i == 1 ? v1 : i == 2 ? v2 : v3), idO,
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
    const int seq = first + row / G, hq = kvh * G + row % G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + C::TO + x * D + lane_base;
    float m_ref = -INFINITY, l = 0.f;
    const int N = soft ? tiles_of(x) : 0;
    if (soft) {
        // Rows are independent through both products: a warp without rows skips the tiles, and what
        // its rows of P hold reaches only its own rows of O, which are never read.
        for (int n = 0; n < (active ? N : 0); ++n) {
            const int e = 2 * x + (n & 1);
            const uint32_t tS = tmem + 64 * e + lane_base;
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
            if (tile_at(x, n) == J - 1 && nlast < BT) {
#pragma unroll
                for (int k = 0; k < BT / 2; ++k) {
                    if (2 * k >= nlast) sv[k].x = -INFINITY;
                    if (2 * k + 1 >= nlast) sv[k].y = -INFINITY;
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
        // q and the ring are idle now: the sums leave through them, written by warps, whole rows a store (rows written
        // to global memory by their threads, 32 lines a store: 11,000 cycles for 256 rows; as a bulk copy a row: 6000)
        float *mine = reinterpret_cast<float *>(smem) + (x * 128 + r) * C::ROW_F;
        const long long prow = ((long long)seq * pp.total_splits + s) * p.Hq + hq;
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
                const float f0 = ex2(m_ref - mu), f1 = ex2(ml.x - mu);
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
                if (rvalid && x == 0)
                    *reinterpret_cast<float2 *>(pp.ml_part + prow * 2) = make_float2(m, l * f0 + ml.y * f1);
                store_rows<C, H>(mine - lane * C::ROW_F + x * H, pp.o_part + x * H, prow * D, min(32, nx - (r - lane)),
                                 lane);
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
            if (rvalid) *reinterpret_cast<float2 *>(pp.ml_part + prow * 2) = make_float2(m_ref, l);
            store_rows<C, D>(mine - lane * C::ROW_F, pp.o_part, prow * D, min(32, nx - (r - lane)), lane);
        }
        if (threadIdx.x == 0 && misc[2]) {
            // a wait gave up: the copies still in flight land (bounded) before the shared memory goes
            (void)mbar_wait(q_full, 0);
            for (int i = max(0, misc[0] - NS); i < misc[0]; ++i) (void)mbar_wait(&k_full[i % NS], (i / NS) & 1);
            for (int i = max(0, misc[1] - NS); i < misc[1]; ++i)
                (void)mbar_wait(&v_full[i % NS], (i / NS) & 1);
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

// Merge of a row's prefix and suffix partials, in that order; W warps a row, warp w taking partials
// w, w + W, ... and the warps' sums added in warp order.  A warp loads NB partials at a time, sums and maxima
// together, and moves its running maximum between batches: one trip to memory for up to NB partials.
template <int D, int W>
__global__ void __launch_bounds__(256) shared_combine_kernel(const SharedParams pp) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int DPV = D / 32, NB = 8;
    __shared__ float red[W > 1 ? 8 : 1][W > 1 ? D + 2 : 1];
    const SplitParams &p = pp.sp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long gw = W == 8 ? (long long)blockIdx.x : (long long)blockIdx.x * 8 + warp;
    const bool live = gw < (long long)p.B * p.Hq;
    const int b = live ? (int)(gw / p.Hq) : 0, hq = live ? (int)(gw - (long long)b * p.Hq) : 0;
    unsigned int flags = 0;
    // The lengths were there before the prefix or suffix kernel read them, and this grid starts after those
    // have: only without them it has to wait first.  (That they can be seen without a wait of this grid's own is the
    // assumption that dap_shared.cuh states.)
    if (pp.total_splits == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    const Span span = seq_span(pp, b, &flags);
    const int np = span.L > 0 && span.P > 0 ? (span.P + pp.prefix_chunk - 1) / pp.prefix_chunk : 0;
    const int n = np + suffix_count(pp, span);
    if (pp.total_splits != 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!live) return;
    if (flags && hq == 0 && lane == 0 && (W == 1 || warp == 0)) flag_error(flags);
    const long long row0 = (long long)b * pp.total_splits * p.Hq + hq;
    float M = -INFINITY, l = 0.f, acc[DPV];
#pragma unroll
    for (int j = 0; j < DPV; ++j) acc[j] = 0.f;
    for (int i0 = W == 1 ? 0 : warp; i0 < n; i0 += NB * W) {
        float x[NB][DPV];
        float2 ml[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = i0 + W * k;
            ml[k] = make_float2(-INFINITY, 0.f);
            if (i < n) {
                const long long row = row0 + (long long)(i < np ? i : i - np + pp.prefix_splits) * p.Hq;
                ml[k] = *reinterpret_cast<const float2 *>(pp.ml_part + row * 2);
                load_row_part<DPV>(pp.o_part + row * D + lane * DPV, x[k]);
            }
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < NB; ++k) m = fmaxf(m, ml[k].x);
        const float mu = m == -INFINITY ? 0.f : m, old = ex2(M - mu);
        M = m;
        l *= old;
#pragma unroll
        for (int j = 0; j < DPV; ++j) acc[j] *= old;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            if (i0 + W * k < n) {
                const float f = ex2(ml[k].x - mu);
                l = fmaf(f, ml[k].y, l);
#pragma unroll
                for (int j = 0; j < DPV; ++j) acc[j] = fmaf(f, x[k][j], acc[j]);
            }
        }
    }
    __nv_bfloat16 *out = p.out + (long long)b * p.o_sb + (long long)hq * p.o_sh;
    if constexpr (W == 1) {
        store_row_part<DPV>(out + lane * DPV, acc, l);
    } else {
#pragma unroll
        for (int j = 0; j < DPV; ++j) red[warp][lane * DPV + j] = acc[j];
        if (lane == 0) {
            red[warp][D] = l;
            red[warp][D + 1] = M;
        }
        __syncthreads();
        if (threadIdx.x < D / 2) {
            const int d = 2 * threadIdx.x;
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < W; ++k) m = fmaxf(m, red[k][D + 1]);
            const float mu = m == -INFINITY ? 0.f : m;
            float a0 = 0.f, a1 = 0.f, ls = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float f = ex2(red[k][D + 1] - mu);
                a0 = fmaf(f, red[k][d], a0);
                a1 = fmaf(f, red[k][d + 1], a1);
                ls = fmaf(f, red[k][D], ls);
            }
            store_out_pair(out + d, a0, a1, ls);
        }
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

// q as [D, Hq, B] with its strides, a box of 64 dims x the G heads of a kv head x 128 / G sequences: 128 rows of
// 128 bytes, in the tile's row order.
bool encode_q_rows(CUtensorMap *map, const SharedArgs &a) {
    const int G = a.Hq / a.Hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.B};
    // a stride over an extent of 1 is never used; give TMA a valid one
    const long long sh = a.Hq > 1 ? a.q_sh : a.D;
    const long long sb = a.B > 1 ? a.q_sb : (long long)a.Hq * sh;
    const cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)sb * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    return encode_bf16(map, a.q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool GATHER>
dap_status launch_prefix(const SharedArgs &a, cudaStream_t stream) {
    using C = PrefixCfg<D, GATHER>;
    const int R = GATHER ? C::BT : gcd_int(a.page_size, C::BT);
    CUtensorMap mq, mk = {}, mv = {};
    if (!encode_q_rows(&mq, a)) return DAP_ERR_CUDA;
    if (!GATHER &&
        (!encode_block_map(&mk, a.k, a.D, a.Hkv, a.page_size, a.num_pages, R, R == C::BT ? C::NBLK : 1) ||
         !encode_block_map(&mv, a.v, a.D, a.Hkv, a.page_size, a.num_pages, R, C::NBLK)))
        return DAP_ERR_CUDA;
    auto kern = shared_prefix_kernel<C>;
    static PerDeviceOcc occ = {};
    if (prepare_kernel(kern, C::THREADS, C::SMEM, &occ, 100) <= 0) return DAP_ERR_CUDA;
    const long long grid = prefix_ctas(a);
    if (grid > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    const SharedParams p = shared_params(a, R);
    const cudaError_t e = launch_dependent_smem(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, mq, mk,
                                                mv, p, a.Hq / a.Hkv);
    return e == cudaSuccess ? DAP_OK : DAP_ERR_CUDA;
}

template <bool GATHER>
dap_status prefix_dims(const SharedArgs &a, cudaStream_t stream) {
    switch (a.D) {
        case 64: return launch_prefix<64, GATHER>(a, stream);
        case 128: return launch_prefix<128, GATHER>(a, stream);
        case 256: return launch_prefix<256, GATHER>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

template <int D>
dap_status combine_d(const SharedArgs &a, cudaStream_t stream) {
    const SharedParams p = shared_params(a, suffix_box_rows(a));
    const long long rows = (long long)a.B * a.Hq;
    if (rows > 0x7FFFFFFFLL) return DAP_ERR_SHAPE;
    // (as launch_combine: a warp per row, or a CTA per row with more than 16 partials)
    const cudaError_t e =
        p.total_splits > 16
            ? launch_dependent(shared_combine_kernel<D, 8>, dim3((unsigned)rows), dim3(256), stream, p)
            : launch_dependent(shared_combine_kernel<D, 1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), stream, p);
    return e == cudaSuccess ? DAP_OK : DAP_ERR_CUDA;
}

}  // namespace

dap_status launch_shared_prefix(const SharedArgs &a, cudaStream_t stream) {
    return a.page_size % 8 != 0 ? prefix_dims<true>(a, stream) : prefix_dims<false>(a, stream);
}

dap_status launch_shared_combine(const SharedArgs &a, cudaStream_t stream) {
    switch (a.D) {
        case 64: return combine_d<64>(a, stream);
        case 128: return combine_d<128>(a, stream);
        case 256: return combine_d<256>(a, stream);
    }
    return DAP_ERR_UNSUPPORTED;
}

bool read_errors_shared_prefix(unsigned int *flags, bool clear) { return read_tu_errors(flags, clear); }

}  // namespace dap
