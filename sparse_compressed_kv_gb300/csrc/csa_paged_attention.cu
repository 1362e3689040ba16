// csa_paged_attention.cu -- shared-KV attention of new tokens over a paged
// cache and the window ring, on the 5th-generation tensor cores:
//   l_j = scale q_h . row_j,   out_h = sum_j softmax_j(l [, sink]) row_j.
//
// A token's row slots are its visible compressed rows, padded to a multiple of
// 8, then its window rows; 48 slots are a chunk.  One kernel of one CTA per SM
// (per 64 heads) divides the chunks of all tokens: each CTA counts every
// token's chunks for itself (the lengths are on the device only), takes an
// equal range of them, and walks it as segments, one per token, through one
// pipeline that does not drain between tokens:
//   warps 0..2    fetch a chunk's rows, 16 each: a group of 8 rows that lies
//                 in one page is one TMA box (64 columns x 8 rows x 8 column
//                 groups: 8 KiB whatever the page size), other groups (page
//                 ends, the last rows, the window) go row by row with 16-byte
//                 cp.async, rows that do not exist as zeros
//   warps 4..7    softmax with a lazily raised maximum
//   warps 8..11   warp 8: Q of the next segment; S = Q . rows^T (M = 64 heads,
//                 N = 48 rows, K = 512), one chunk ahead of warp 9: O^T +=
//                 rows^T . P^T (M = 128 columns a tile, N = 64 heads); all
//                 four: a segment's epilogue, tile by tile, while the next
//                 segment's rows, logits and weights are on their way (its
//                 first O^T product takes each tile as it is drained)
// A group's 8 KiB hold 8 column groups of 8 rows x 128 bytes (the swizzle
// atom), so the same bytes are the K-major operand of S (row groups 8 KiB
// apart) and the MN-major operand of O^T (column groups 1 KiB apart, row
// groups 8 KiB).
//
// A segment that is a whole token writes the output; the parts of a token cut
// between CTAs go to the workspace as (O, m, l) and a second kernel joins
// them.  The accumulator of tcgen05 drops bits below its last place, so
// sums of thousands of rows drift; at least every kFlush chunks O^T is added,
// rounded, into the CTA's own f32 partial and starts again from zero.
//
// Bound by (times replayed from a graph): DRAM where a CTA has tens of chunks (32 ragged contexts, 545 MB,
// 103 us; one million tokens at ratio 4, 269 MB, 58 us); with two terms of P
// the products and the turn of a stage (2,070 cycles a chunk); by its latency
// chain where a CTA has one or two (8,192 rows 14.8 us, 256 rows 9.1 us, join
// included; called in a stream 14.6 and 9.5).  A stage's turn (released, copied, logits, weights, products) takes
// 5,500 cycles, so the stages set the pace: three of 48 rows instead of two of
// 64, what fits beside Q, take 2,760 cycles per 64 rows instead of 3,780 with
// two terms and 2,840 instead of 3,130 with one (128-head drafts 82.5 -> 76.7
// us, 256 tokens of 1K rows 72.6 -> 68.1; one token of 8,192 rows, two rounds
// before and three now, 14.0 -> 14.8), and need no prefetch into L2 (with it: 105
// instead of 103 us).  Chunks of 32 rows would pay the instructions' floor of 26 to
// 33 cycles twice as often.
#include <math.h>

#include <type_traits>

#include "csa_paged_attention.cuh"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kSmThreads = 128;                 // warps 4..7
constexpr int kChunk = 48;
constexpr int kSlices = kChunk / 16;            // of 16 rows: one K step of O^T each
constexpr int kQBytes = kHG * kHD * 2;          // 64 KiB
constexpr int kGroupBytes = 8 * kHD * 2;        // 8 rows: 8 KiB
constexpr int kStageBytes = kChunk / 8 * kGroupBytes;   // 48 KiB
constexpr int kStages = 3;
constexpr int kPBytes = kHG * kChunk * 2;       // one bf16 term of P: 6 KiB
constexpr int kStagedHeads = 16;                // of a bf16 output, on their way through shared memory
template <int kTerms>
constexpr int kStagedBytes = kTerms == 1 ? 4 * staged_bytes(kStagedHeads) : 0;
constexpr int kSCol = 0;                        // two S buffers of 64 columns
constexpr int kOCol = 128;                      // O^T: 4 tiles x 64 heads
constexpr uint32_t kTmemCols = 512;
// With two terms of P, the first two tiles take both from one reading of the
// rows (N = 128: hi's sums, then lo's) into 64 columns each; tensor memory has
// room for no more.
template <int kTerms>
constexpr int kWide = kTerms == 2 ? 2 : 0;
template <int kTerms>
__device__ __forceinline__ constexpr uint32_t o_col(int dd) {
    return kOCol + kHG * (dd + (dd < kWide<kTerms> ? dd : kWide<kTerms>));
}
constexpr int kMaxRec = 64;                     // segments a CTA lists at a time
constexpr int kSegCost = 4;                     // a segment's epilogue, in chunks (3: 128 contexts of 512 rows 30.3
                                                // us instead of 29.3; 2: 128-head drafts 82.5 instead of 76.5)
// Chunks a token may exceed the mean before tokens are cut.  (240 rows; 2 and 3
// chunks measure the same within 0.5%.  At 8 chunks 64 tokens of 512 rows gain, 27.6
// -> 26.4 us, and one of 256 rows loses, 9.4 -> 15.4.  At 16, 150 tokens of 250 to 500
// rows gain, 30.8 -> 26.6 us, and 64 of 512 rows, 27.6 -> 23.4, but 64 of 512 to 1,024
// rows lose, 27.9 -> 34.3, 128 of 32 to 1,024 rows, 31.4 -> 46.3, and one of 600, 9.0 ->
// 22.8.)
constexpr int kCutAbove = 5;
constexpr int kFlushF32 = 53, kFlushBf16 = 682; // chunks between roundings of the accumulator, at most

struct Smem {
    uint64_t q_full, q_free;
    uint64_t full[kStages], empty[kStages][kSlices];   // a stage is released 16 rows at a time
    uint64_t sfull[2], sfree[2];
    uint64_t pfull[2], pfree;    // P's rows 0..15 and 32..47, then 16..31
    uint64_t stretch[2], stretch_free[2];   // the factors of a stretch are written, used
    uint64_t ofree[4];           // a tile of O^T is drained
    uint32_t tmem_holder;
    uint32_t maskw[kStages][kSlices];
    uint32_t flag[2][4];
    float alpha[kHG];
    alignas(16) float fin[2][kHG];     // of a stretch: factors of the output,
    alignas(16) float flush[2][kHG];   // and of the partial so far
    WorkSmem<kMaxRec> work;
};

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                            int32_t z, int32_t w, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar)),
        "l"(policy)
        : "memory");
}

// tmem_ld16x2_raw's lanes, at columns c .. and c + 8 .. (8 each)
__device__ __forceinline__ void tmem_ld8x2_raw(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
}

// kTerms: bf16 terms of P (2 for an f32 output, 1 for bf16).
template <int kTerms>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_rows, const PagedArgs A) {
    constexpr int kFlush = kTerms == 2 ? kFlushF32 : kFlushBf16;
    constexpr int kPieceBytes = kTerms * kHG * 16;       // 8 rows of P
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem<1024>(smem_raw);
    uint8_t *sQ = smem;
    uint8_t *sRows = sQ + kQBytes;                       // [stage][6 groups][8 col groups][8 rows][128 B]
    uint8_t *sP = sRows + kStages * kStageBytes;         // [8 rows of the chunk][term][64 heads][16 B]
    uint8_t *sOut = sP + kTerms * kPBytes;               // [epilogue warp][16 heads][32 columns], bf16 output
    Smem &S = *reinterpret_cast<Smem *>(sOut + kStagedBytes<kTerms>);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = blockIdx.y, h0 = hg * kHG;
    const int H = A.H;

    if (tid == 0) {
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_free, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&S.full[i], kSlices);
            for (int k = 0; k < kSlices; ++k) mbar_init(&S.empty[i][k], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.sfree[i], kSmThreads);
        }
        mbar_init(&S.pfull[0], kSmThreads);
        mbar_init(&S.pfull[1], kSmThreads);
        mbar_init(&S.pfree, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.stretch[i], kSmThreads);
            mbar_init(&S.stretch_free[i], kEpThreads);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&S.ofree[i], kEpThreads);
        mbar_fence_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_rows);
    }
    if (warp == 8) {
        tmem_alloc(&S.tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();

    Work<kThreads, kMaxRec, kChunk, kSegCost, kCutAbove> W(A, S.work);
    W.count();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_holder;
    W.divide();
    W.first_list();
    const int ndt = W.ndt, dt0 = W.dt0;                          // 128-column tiles of this CTA
    const Rec *const rec = S.work.rec;

    // pipeline positions, kept across lists of segments
    uint32_t n_fetch = 0;                // chunks fetched
    uint32_t nq = 0, np = 0;             // chunks whose S / O^T product was issued
    uint32_t n_ql = 0;                   // Q loads issued
    uint32_t n_sm = 0;                   // chunks through the softmax; whose O^T product was issued
    uint32_t n_ep = 0;                   // stretches through the softmax, the epilogue

    for (;;) {
        __syncthreads();
        W.advance();
        const int nrec = S.work.nrec;
        const bool more = S.work.more != 0;
        if (nrec == 0) break;

        if (warp >= 8) {
            // -------------------------------------------- products, epilogue
            // Step j: warp 8 issues S of chunk j, warp 9 O^T of chunk j - 1, and
            // all four drain O^T where that chunk ends a stretch.  A whole
            // warp keeps step and one elected thread issues: a 64 x 64 x 16
            // instruction every 33 cycles behind elect.sync, every 54 behind
            // `lane == 0`.
            constexpr uint32_t id_qk = idesc_bf16<kHG, kChunk, false>();
            constexpr uint32_t id_pv = idesc_bf16<128, kHG, true>(), id_wide = idesc_bf16<128, 2 * kHG, true>();
            const uint64_t q_desc = sw128_desc(smem_addr(sQ), 16, 1024);
            const uint64_t r_desc = sw128_desc(smem_addr(sRows), 16, kGroupBytes);
            const uint64_t a_desc = sw128_desc(smem_addr(sRows) + 2 * dt0 * 1024, 1024, kGroupBytes);
            const uint64_t p_desc = atom_desc(smem_addr(sP), kPieceBytes, 128);
            const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int hmax = min(kHG, H - h0);
            // slices of 16 rows (0 and 2, then 1), each released when its products are done
            auto product = [&](int dd, int ks, uint64_t ad, uint32_t acc) {
                const uint64_t av = ad + off(2 * dd * 1024 + ks * 2 * kGroupBytes);
                const uint32_t d = tmem + o_col<kTerms>(dd);
                const uint64_t pd = p_desc + off(2 * ks * kPieceBytes);
                if (dd < kWide<kTerms>) {
                    umma_bf16(d, av, pd, id_wide, acc);
                } else {
                    umma_bf16(d, av, pd, id_pv, acc);
                    if (kTerms == 2) umma_bf16(d, av, pd + off(kHG * 16), id_pv, 1u);
                }
            };
            auto pv = [&](auto ntile, uint64_t ad, int st, int k0) {
#pragma unroll
                for (int ks = k0; ks < kSlices; ks += 2) {
#pragma unroll
                    for (int dd = 0; dd < ntile; ++dd) product(dd, ks, ad, 1u);
                    umma_commit(&S.empty[st][ks]);
                }
                if (k0 == 1) umma_commit(&S.pfree);
            };
            int i = 0, k = 0, nch = 0, every = 1, z = 0;     // chunk j: k of segment i, z of a stretch
            auto settle = [&]() {
                while (i < nrec) {
                    nch = rec[i].c1 - rec[i].c0;
                    if (nch > 0) break;
                    ++i;
                }
                k = z = 0;
                if (i < nrec) every = flush_every<kFlush>(nch);
            };
            settle();
            int bi = -1, bk = 0, bz = 0, bn = 0, be = 1;     // the chunk before it
            for (;;) {
                if (warp == 8 && i < nrec) {
                    if (k == 0) {
                        // the last product of the segment before is done with Q
                        if (n_ql > 0) mbar_wait(&S.q_free, (n_ql - 1) & 1u, A.status);
                        __syncwarp();
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&S.q_full, kQBytes);
                            tma_load_4d(sQ, &tm_q, 0, h0, 0, rec[i].t, &S.q_full, policy_evict_normal());
                        }
                        __syncwarp();
                        mbar_wait(&S.q_full, n_ql & 1u, A.status);
                        ++n_ql;
                    }
                    const int st = nq % kStages, sb = nq & 1u;
                    mbar_wait(&S.full[st], (nq / kStages) & 1u, A.status);
                    mbar_wait(&S.sfree[sb], ((nq >> 1) & 1u) ^ 1u, A.status);
                    ++nq;
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t rd = r_desc + off(st * kStageBytes);
                        const uint32_t d = tmem + kSCol + sb * 64;
#pragma unroll
                        for (int kk = 0; kk < 32; ++kk) {
                            const uint32_t cg = kk >> 2, ko = (kk & 3) * 32;
                            umma_bf16(d, q_desc + off(cg * (kHG * 128) + ko), rd + off(cg * 1024 + ko), id_qk,
                                      kk > 0 ? 1u : 0u);
                        }
                        umma_commit(&S.sfull[sb]);
                        if (k + 1 == nch) umma_commit(&S.q_free);
                    }
                    __syncwarp();
                }
                if (warp == 9 && bi >= 0) {
                    const int st = np % kStages;
                    const uint32_t pp = np & 1u;
                    mbar_wait(&S.pfull[0], pp, A.status);
                    ++np;
                    const uint64_t ad = a_desc + off(st * kStageBytes);
                    if (bz == 0) {
                        mbar_wait(&S.pfull[1], pp, A.status);
                        // a stretch's first chunk, tile by tile as the stretch
                        // before it leaves tensor memory
                        for (int dd = 0; dd < ndt; ++dd) {
                            if (n_ep > 0) mbar_wait(&S.ofree[dd], (n_ep - 1) & 1u, A.status);
                            __syncwarp();
                            tc_fence_after();
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < kSlices; ++ks) product(dd, ks, ad, ks > 0 ? 1u : 0u);
                                if (dd + 1 == ndt) {
                                    for (int ks = 0; ks < kSlices; ++ks) umma_commit(&S.empty[st][ks]);
                                    umma_commit(&S.pfree);
                                }
                            }
                            __syncwarp();
                        }
                    } else {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (half == 1) mbar_wait(&S.pfull[1], pp, A.status);
                            __syncwarp();
                            tc_fence_after();
                            if (elect_one()) {
                                if (ndt == 4) pv(std::integral_constant<int, 4>{}, ad, st, half);
                                else if (ndt == 2) pv(std::integral_constant<int, 2>{}, ad, st, half);
                                else pv(std::integral_constant<int, 1>{}, ad, st, half);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (bi >= 0) {
                    ++n_sm;
                    if (bk + 1 == bn || bz + 1 == be) {
                        // ---- O^T into the partial, or the output
                        const int t = rec[bi].t, flags = rec[bi].flags;
                        const int64_t obase = (static_cast<int64_t>(t) * H + h0) * kHD;
                        const int64_t pslot = static_cast<int64_t>(rec[bi].slot) * gridDim.y + hg;
                        const int e = n_ep & 1u;
                        (void)CSA_CHECK(rec[bi].slot < 2 * W.G && t < W.T, A.status);
                        const bool add = bk >= be;               // the partial holds earlier stretches
                        const bool part = (flags & kRecPart) || bk + 1 < bn;
                        mbar_wait(&S.stretch[e], (n_ep >> 1) & 1u, A.status);
                        mbar_wait(&S.pfree, (n_sm - 1) & 1u, A.status);   // its last product
                        ++n_ep;
                        __syncwarp();
                        tc_fence_after();
                        drain_stretch<kTerms == 1, kWide<kTerms>, kStagedHeads>(
                            A, tmem + lane_off + kOCol, S.fin[e], S.flush[e], S.ofree, sOut + (warp & 3) * staged_bytes(kStagedHeads), dt0,
                            ndt, 0, kHG, hmax, obase, pslot,
                            add, part);
                        mbar_arrive(&S.stretch_free[e]);
                        __syncwarp();
                    }
                }
                if (i >= nrec) break;
                bi = i, bk = k, bz = z, bn = nch, be = every;
                z = z + 1 == every ? 0 : z + 1;
                if (++k == nch) {
                    ++i;
                    settle();
                }
            }
        } else if (warp < kSlices) {
            // -------------------------------------------- row fetch
            // The warp walks the list's chunks, 16 rows of each.  Lane l (and
            // l + 16) looks after row l; three chunks before it is copied its page
            // number is on its way from the table, two before it is a row of
            // the pool.
            const int li = warp;
            const int rl = lane & 15;
            int bad = 0;
            struct Cursor {
                int i, c;
            };
            auto settle = [&](Cursor &k) {             // to the next segment that has chunks
                while (k.i < nrec && k.c >= rec[k.i].c1) {
                    ++k.i;
                    if (k.i < nrec) k.c = rec[k.i].c0;
                }
            };
            auto advance = [&](Cursor &k) {
                ++k.c;
                settle(k);
            };
            struct Entry {
                int32_t page, in_page;                 // in_page < 0: not a row of the pool
                bool box;                              // 8 rows of one page from here on
            };
            auto look_up = [&](const Cursor &k) {
                Entry e{-1, -1, false};
                if (k.i >= nrec) return e;
                const int n = rec[k.i].n, j = k.c * kChunk + 16 * li + rl;
                if (j < n) {
                    const int pg = static_cast<int>(A.page_div.div(j));
                    e.in_page = j - pg * A.L.page_rows;
                    e.page = A.L.table[static_cast<int64_t>(rec[k.i].b) * A.L.max_pages + pg];
                    e.box = j + 8 <= n && e.in_page + 8 <= A.L.page_rows;
                }
                return e;
            };
            struct Place {
                int32_t row;                           // row of the pool, or -1
                uint32_t box;                          // bit g: group g of 8 rows is one box
            };
            auto place = [&](const Entry &e) {
                Place p{-1, 0};
                if (e.in_page >= 0) {
                    if (e.page < 0 || e.page >= A.num_pages) bad |= CSA_DEV_BAD_INDEX;
                    else p.row = static_cast<int32_t>(e.page * A.page_stride) + e.in_page;
                    if (!CSA_CHECK(p.row < A.total_rows, A.status)) p.row = -1;
                }
                const uint32_t bx = __ballot_sync(0xffffffffu, e.box);
                p.box = (bx & 1u) | (bx >> 7 & 2u);
                return p;
            };
            int pending = -1;                          // stage whose cp.async rows are in flight
            auto land = [&](bool newer) {              // ... have landed: hand the stage over
                if (newer) cp_async_wait<1>();
                else cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.full[pending]);
                pending = -1;
            };
            // rows are read once, or once by each of two groups of heads
            const uint64_t pol = gridDim.y > 1 ? policy_evict_normal() : policy_evict_first();
            Cursor cur{0, rec[0].c0};
            settle(cur);
            Cursor far = cur;
            const Entry e0 = look_up(far);
            advance(far);
            const Entry e1 = look_up(far);
            advance(far);
            Entry ahead = look_up(far);
            Place now = place(e0), next = place(e1);
            while (cur.i < nrec) {
                const Rec &r = rec[cur.i];
                const int j0 = cur.c * kChunk + 16 * li, wslot = rec_window_slot(r);
                const __nv_bfloat16 *src = nullptr;
                if (now.row >= 0) {
                    src = A.cache + static_cast<int64_t>(now.row) * kHD;
                } else if (r.near > 0 && j0 + rl >= wslot && j0 + rl - wslot < r.near) {
                    const int64_t x = r.first + (j0 + rl - wslot);
                    if (x < r.first_res) bad |= CSA_DEV_MISSING_SWA;
                    else
                        src = static_cast<const __nv_bfloat16 *>(A.L.swa_kv) +
                              (static_cast<int64_t>(r.b) * A.L.swa_cap + A.swa_div.mod64(x)) * kHD;
                }
                const uint32_t okm = __ballot_sync(0xffffffffu, src != nullptr) & 0xFFFFu;
                const int32_t y1 = __shfl_sync(0xffffffffu, now.row, 8);
                const int st = n_fetch % kStages;
                const uint32_t ph = ((n_fetch / kStages) & 1u) ^ 1u;
                if (pending >= 0 && !__all_sync(0xffffffffu, mbar_test_wait(&S.empty[st][li], ph))) land(false);
                mbar_wait(&S.empty[st][li], ph, A.status);
                __syncwarp();
                uint8_t *rows = sRows + st * kStageBytes + 2 * li * kGroupBytes;
                if (lane == 0) {
                    S.maskw[st][li] = okm;
                    if (now.box) {
                        // (a bad page: a box behind the pool reads as zeros)
                        mbar_expect_tx(&S.full[st], (now.box == 3u ? 2 : 1) * kGroupBytes);
                        if (now.box & 1u)
                            tma_load_3d(rows, &tm_rows, 0, now.row >= 0 ? now.row : A.total_rows, 0, &S.full[st], pol);
                        if (now.box & 2u)
                            tma_load_3d(rows + kGroupBytes, &tm_rows, 0, y1 >= 0 ? y1 : A.total_rows, 0, &S.full[st], pol);
                    }
                }
                const bool by_row = now.box != 3u;
                if (by_row) {
#pragma unroll 1
                    for (int g = 0; g < 2; ++g) {
                        if (now.box >> g & 1u) continue;
#pragma unroll
                        for (int rr = 0; rr < 8; ++rr) {
                            const __nv_bfloat16 *p = reinterpret_cast<const __nv_bfloat16 *>(__shfl_sync(
                                0xffffffffu, reinterpret_cast<unsigned long long>(src), 8 * g + rr));
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int k = lane + 32 * u;   // 16-byte piece of the row
                                cp_async16(rows + g * kGroupBytes + (k >> 3) * 1024 + rr * 128 + (((k & 7) ^ rr) << 4),
                                           p ? static_cast<const void *>(p + k * 8) : A.cache, p != nullptr);
                            }
                        }
                    }
                    cp_async_commit();
                }
                // the queue moves up
                now = next;
                next = place(ahead);
                advance(far);
                ahead = look_up(far);
                advance(cur);
                if (pending >= 0) land(by_row);
                if (by_row) pending = st;
                else if (lane == 0) mbar_arrive(&S.full[st]);
                ++n_fetch;
            }
            if (pending >= 0) land(false);
            bad = static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad)));
            if (lane == 0 && W.lead) raise_status(A.status, bad);
        } else if (warp >= 4) {
            // -------------------------------------------- softmax
            const int q = warp & 3;                  // TMEM lane quarter
            const int hl = q * 16 + (lane & 15);     // head of this lane (two lanes per head)
            const bool upper = lane >= 16;           // rows 32..47 and 24..31 of the chunk, others 0..23
            const bool hv = h0 + hl < H;
            const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
            for (int i = 0; i < nrec; ++i) {
                const int nch = rec[i].c1 - rec[i].c0;
                if (nch <= 0) {
                    if (rec[i].flags & kRecZero) {
                        const int64_t obase = (static_cast<int64_t>(rec[i].t) * H + h0) * kHD;
                        for (int x = tid - 128; x < min(kHG, H - h0) * 128 * ndt; x += kSmThreads) {
                            const int64_t at = obase + (x / (128 * ndt)) * kHD + dt0 * 128 + x % (128 * ndt);
                            if (kTerms == 1) static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(0.f);
                            else static_cast<float *>(A.out)[at] = 0.f;
                        }
                    }
                    continue;
                }
                const bool cut = rec[i].flags & kRecPart;
                float m_ref = -INFINITY, l = 0.f, m_flush = -INFINITY;
                const int every = flush_every<kFlush>(nch);
                for (int k = 0, z = 0; k < nch; ++k, ++n_sm, z = z + 1 == every ? 0 : z + 1) {
                    const int st = n_sm % kStages, sb = n_sm & 1u;
                    // (a wait's lanes may leave it at different polls; what is
                    // .aligned below, tensor memory and barriers, wants the warp whole)
                    mbar_wait(&S.sfull[sb], (n_sm >> 1) & 1u, A.status);
                    __syncwarp();
                    tc_fence_after();
                    uint32_t sr[16], sr2[8];
                    tmem_ld16x2_raw(tmem + lane_off + kSCol + sb * 64, sr);
                    tmem_ld8x2_raw(tmem + lane_off + kSCol + sb * 64 + 16, sr2);
                    tmem_wait_ld();
                    tc_fence_before();
                    mbar_arrive(&S.sfree[sb]);
                    mbar_wait(&S.full[st], (n_sm / kStages) & 1u, A.status);   // orders the mask words
                    const uint32_t mw[kSlices] = {S.maskw[st][0], S.maskw[st][1], S.maskw[st][2]};
                    // Every row real and a scale >= 0: the maximum of the raw
                    // logits, the scale in the exponent's fma.  Otherwise
                    // scaled logits, rows that do not exist at -inf.
                    float x[24];
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    float xs = 1.f;
                    if ((mw[0] & mw[1] & mw[2]) == 0xFFFFu && A.scale_log2 >= 0.f) {
                        xs = A.scale_log2;
#pragma unroll
                        for (int j = 0; j < 24; ++j) {
                            x[j] = __uint_as_float(j < 16 ? sr[j & 15] : sr2[j & 7]);
                            mq[j & 3] = fmaxf(mq[j & 3], x[j]);
                        }
                    } else {
                        const uint32_t mh = (upper ? mw[2] : mw[0]) | (mw[1] >> (upper ? 8 : 0) & 0xFFu) << 16;
#pragma unroll
                        for (int j = 0; j < 24; ++j) {
                            const uint32_t v = j < 16 ? sr[j & 15] : sr2[j & 7];
                            x[j] = ((mh >> j) & 1u) ? __uint_as_float(v) * A.scale_log2 : -INFINITY;
                            mq[j & 3] = fmaxf(mq[j & 3], x[j]);
                        }
                    }
                    float mc = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                    mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 16)) * xs;
                    // a head whose maximum rises by more than kRescaleAbove rescales
                    // what has been accumulated
                    const bool need = hv && m_ref != -INFINITY && mc > m_ref + kRescaleAbove;
                    const uint32_t wneed = __ballot_sync(0xffffffffu, need);
                    if (lane == 0) S.flag[sb][q] = wneed;
                    float alpha = 1.f;
                    if (need) {
                        alpha = exp2f(m_ref - mc);
                        m_ref = mc;
                        l *= alpha;
                    } else if (m_ref == -INFINITY) {
                        m_ref = mc;
                    }
                    __syncwarp();
                    named_bar_sync(kBarSm, kSmThreads);
                    const bool any = (S.flag[sb][0] | S.flag[sb][1] | S.flag[sb][2] | S.flag[sb][3]) != 0;
                    if (any && z != 0) {
                        if (!upper) S.alpha[hl] = alpha;
                        mbar_wait(&S.pfree, (n_sm - 1) & 1u, A.status);   // the product before this one
                        __syncwarp();
                        named_bar_sync(kBarSm, kSmThreads);
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < static_cast<int>(o_col<kTerms>(ndt) - kOCol); x += 16) {
                            uint32_t o[16];
                            const uint32_t ta2 = tmem + lane_off + kOCol + x;
                            tmem_ld16_raw(ta2, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * S.alpha[x % kHG + e]);
                            tmem_st16(ta2, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        named_bar_sync(kBarSm, kSmThreads);
                    }
                    // P = 2^(x - m_ref), rounded to bf16 (one term: the sum
                    // is that of the rounded weights, so they add up to 1) or as
                    // hi + lo with lo the rounded rest
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref;
                    float sq[2] = {0.f, 0.f};
                    uint8_t *const pr = sP + hl * 16;
                    // two thirds of the lane's rows, then the rest: the first products
                    // start under the rest's exponentials
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t phi[8], plo[8];
#pragma unroll
                        for (int u = 0; u < (half == 0 ? 8 : 4); ++u) {
                            const int j = 16 * half + 2 * u;
                            const float p0 = fast_exp2(fmaf(x[j], xs, -mr));
                            const float p1 = fast_exp2(fmaf(x[j + 1], xs, -mr));
                            const uint32_t hi = pack_bf16x2(p0, p1);
                            const float g0 = __uint_as_float(hi << 16), g1 = __uint_as_float(hi & 0xFFFF0000u);
                            phi[u] = hi;
                            if (kTerms == 2) {
                                sq[u & 1] += p0 + p1;
                                plo[u] = pack_bf16x2(p0 - g0, p1 - g1);
                            } else {
                                sq[u & 1] += g0 + g1;
                            }
                        }
                        if (half == 0 && n_sm > 0) mbar_wait(&S.pfree, (n_sm - 1) & 1u, A.status);
#pragma unroll
                        for (int e = 0; e < (half == 0 ? 2 : 1); ++e) {
                            const int piece = half == 0 ? (upper ? 4 : 0) + e : (upper ? 3 : 2);
                            uint8_t *const at = pr + piece * kPieceBytes;
                            *reinterpret_cast<uint4 *>(at) = make_uint4(phi[4 * e], phi[4 * e + 1], phi[4 * e + 2], phi[4 * e + 3]);
                            if (kTerms == 2)
                                *reinterpret_cast<uint4 *>(at + kHG * 16) =
                                    make_uint4(plo[4 * e], plo[4 * e + 1], plo[4 * e + 2], plo[4 * e + 3]);
                        }
                        fence_proxy_async_smem();
                        mbar_arrive(&S.pfull[half]);
                    }
                    const float sum = sq[0] + sq[1];
                    l += sum + __shfl_xor_sync(0xffffffffu, sum, 16);

                    const bool last = k + 1 == nch;
                    if (!last && z + 1 != every) continue;
                    // the stretch's factors for the epilogue
                    const int e = n_ep & 1u;
                    mbar_wait(&S.stretch_free[e], ((n_ep >> 1) & 1u) ^ 1u, A.status);
                    ++n_ep;
                    if (!upper) {
                        S.flush[e][hl] = m_flush == -INFINITY ? 1.f : exp2f(m_flush - m_ref);
                        float f = 1.f;
                        if (last && !cut) {
                            float zs = l;
                            if (A.sinks && hv) zs += exp2f(A.sinks[h0 + hl] * kLog2e - m_ref);
                            f = m_ref == -INFINITY ? 0.f : 1.f / zs;     // (a sink of NaN: NaN)
                        }
                        S.fin[e][hl] = f;
                        if (last && cut && dt0 == 0)
                            A.part_ml[(static_cast<int64_t>(rec[i].slot) * gridDim.y + hg) * kHG + hl] =
                                make_float2(m_ref, l);
                    }
                    m_flush = m_ref;
                    mbar_arrive(&S.stretch[e]);
                }
            }
        }
        if (!more) break;
        __syncthreads();                 // the list is done with
        if (tid == 0) {
            S.work.nrec = 0;
            S.work.more = 0;
        }
        W.next_list();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int kTerms>
size_t smem_bytes() { return 1024 + kQBytes + kStages * kStageBytes + kTerms * kPBytes + kStagedBytes<kTerms> + sizeof(Smem); }

}  // namespace

size_t paged_attention_workspace(const csa_paged_layout_t &, const csa_params_t &p) {
    return ws_plan(p).total;
}

cudaError_t launch_paged_attention(const Launch &lc, const csa_paged_layout_t &L,
                                   const csa_params_t &p, const void *cache, int64_t num_pages,
                                   int64_t page_stride, const void *q, const float *sinks,
                                   csa_type_t out_type, void *out, int32_t *status, void *ws) {
    const int H = p.n_heads, groups = groups_of(p);
    const int64_t total_rows = paged_rows(L, num_pages, page_stride);
    CUtensorMap tq, tr;
    {
        // [64 columns][heads][8 column groups][tokens]
        const uint64_t dims[4] = {64, static_cast<uint64_t>(H), 8, static_cast<uint64_t>(L.num_tokens)};
        const uint64_t strides[3] = {kHD * 2, 128, static_cast<uint64_t>(H) * kHD * 2};
        const uint32_t box[4] = {64, kHG, 8, 1};
        if (encode_tensor_map_bf16(&tq, q, 4, dims, strides, box) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    {
        // [64 columns][rows of the pool][8 column groups]
        const uint64_t dims[3] = {64, static_cast<uint64_t>(total_rows), 8};
        const uint64_t strides[2] = {kHD * 2, 128};
        const uint32_t box[3] = {64, 8, 8};
        if (encode_tensor_map_bf16(&tr, cache, 3, dims, strides, box) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    PagedArgs A = paged_args(lc, L, p, num_pages, page_stride, sinks, out_type, out, status, ws);
    A.cache = static_cast<const __nv_bfloat16 *>(cache);
    const int ctas = static_cast<int>(A.split_div[0].d);
    cudaError_t e;
    if (A.bf16_out) {
        e = prepare_kernel<paged_attention_kernel<1>>(smem_bytes<1>());
        if (e == cudaSuccess)
            e = launch_pdl(paged_attention_kernel<1>, dim3(ctas, groups), dim3(kThreads), smem_bytes<1>(), lc.stream, tq, tr, A);
    } else {
        e = prepare_kernel<paged_attention_kernel<2>>(smem_bytes<2>());
        if (e == cudaSuccess)
            e = launch_pdl(paged_attention_kernel<2>, dim3(ctas, groups), dim3(kThreads), smem_bytes<2>(), lc.stream, tq, tr, A);
    }
    if (e != cudaSuccess) return e;
    // no token can be cut: nothing to join
    const int64_t slots_max = (static_cast<int64_t>(L.max_pages) * L.page_rows + 7) / 8 * 8 + p.window;
    if (slots_max <= kCutAbove * kChunk) return cudaSuccess;
    const int entries = L.num_tokens < ctas ? L.num_tokens : ctas;
    // one long context is cut into many parts, a batch's tokens into few
    return A.bf16_out ? launch_join<true>(lc, A, entries, groups, slots_max)
                      : launch_join<false>(lc, A, entries, groups, slots_max);
}

}  // namespace csa
