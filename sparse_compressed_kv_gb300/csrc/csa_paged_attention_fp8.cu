// csa_paged_attention_fp8.cu -- shared-KV attention of new tokens over a paged
// cache of e4m3 rows and their window ring, on the 5th-generation tensor cores:
//   l_j = scale q_h . (s_j c_j),   out_h = sum_j softmax_j(l [, sink]) s_j c_j.
//
// The division of the work, the segments, the partials and the joins are those
// of the bf16 rows' kernel (csa_paged_attention.cuh); a chunk is 64 row slots, and
// the codes are the tensor cores' operands as they lie in memory:
//   warps 0..3    fetch a chunk's rows, 16 each: 8 rows of one page are one TMA box
//                 (128 columns x 8 rows x 4 column groups: 4 KiB), others go row
//                 by row with 16-byte cp.async; and each row's scale
//   warps 4..7    the query, 16 heads each, split in two e4m3 terms where a segment
//                 begins; softmax with a lazily raised maximum
//   warps 8..11   warp 8: S = Q . rows^T (M = 64 heads x 2 terms, N = 64 rows, K =
//                 512), one chunk ahead of warp 9: O^T += rows^T . P^T (M = 128
//                 columns a tile, N = 64 heads, K = 64 rows); all four: a segment's
//                 epilogue
// A group's 4 KiB hold 4 column groups of 8 rows x 128 bytes (the swizzle atom):
// the K-major operand of S and the MN-major operand of O^T.
//
// Q = hi + lo: a head's largest magnitude is brought to [2^7, 2^8) by a power of
// two; hi is the nearest e4m3 value, lo the nearest to what is left.  A bf16
// number has 8 bits and each term takes 4, so the two are exact down to 2^-10 of
// the largest (lo's last place is 2^-9).  Rows 32 q + i and 32 q + 16 + i of the
// operand are the terms of head 16 q + i, so that both sums lie in the same warp's
// quarter of tensor memory, and the softmax adds them.
//
// P = 2^(l_j - m) s_j as e5m2 terms of 3 bits: what f16 rounds it to, cut into
// bytes (e5m2 is f16's upper byte), three terms for a bf16 output (2^-9), six for
// f32 (2^-18).  e4m3 would hold 4 bits a term, but 18 powers of two; e5m2 holds 32:
// with the maximum m of l_j + log2 s_j brought to 2^7 (and up to 2^15 before it is
// raised) a weight is cut off below 2^-24 of the largest, so that ten thousands of
// small weights keep their sum.
#include <cuda_fp16.h>

#include <type_traits>

#include "csa_fp8.cuh"
#include "csa_paged_attention.cuh"

namespace csa {
namespace {

constexpr int kChunk = 64;
constexpr int kSlices = kChunk / 16;            // of 16 rows, one per fetch warp
constexpr int kSteps = kChunk / 32;             // of 32 rows: one K step of O^T each
constexpr int kQBytes = 2 * kHG * kHD;          // 64 KiB
constexpr int kGroupBytes = 8 * kHD;            // 8 rows: 4 KiB
constexpr int kStageBytes = kChunk / 8 * kGroupBytes;   // 32 KiB
constexpr int kStages = 4;
constexpr int kTermBytes = kHG * 16;            // 16 rows of a term of P
template <int kTerms>
constexpr int kPieceBytes = kTerms * kTermBytes;
template <int kTerms>
constexpr int kStagedBytes = kTerms == 3 ? 4 * kOutBytes : 0;
constexpr int kSCol = 0;                        // two S buffers of 64 columns
constexpr int kOCol = 128;                      // O^T: 4 tiles x 64 heads
constexpr uint32_t kTmemCols = 512;
// The first two tiles take two terms from one reading of the rows (N = 128: 64.6
// cycles instead of twice 48.3) into 64 columns each; tensor memory has room for
// no more.
constexpr int kWide = 2;
__device__ __forceinline__ constexpr uint32_t o_col(int dd) { return kOCol + kHG * (dd + (dd < kWide ? dd : kWide)); }
constexpr int kSegCost = 3;                     // a segment's epilogue, in chunks
constexpr int kCutAbove = 4;                    // chunks a token may exceed the mean before tokens are cut
constexpr int kFlushF32 = 27, kFlushBf16 = 341; // chunks between roundings of the accumulator, at most
constexpr float kTop = 7.f;                     // log2 of the weight that the maximum is brought to

struct PagedFp8Args : PagedArgs {
    const uint8_t *codes;
    const float *scales, *swa_scales;
    int64_t scale_stride;
    const __nv_bfloat16 *q;
};

struct Smem {
    uint64_t q_full;
    uint64_t full[kStages], empty[kStages][kSteps];    // a stage is released 32 rows at a time
    uint64_t sfull[2], sfree[2];
    uint64_t pfull[kSteps], pfree;
    uint64_t stretch[2], stretch_free[2];   // the factors of a stretch are written, used
    uint64_t ofree[4];           // a tile of O^T is drained
    uint32_t tmem_holder;
    uint32_t maskw[kStages][kSlices];
    uint32_t flag[2][4];
    float alpha[kHG];
    alignas(16) float scale[kStages][kChunk];   // of a row (absent rows: 0),
    alignas(16) float scale_log[kStages][kChunk];   // and its logarithm
    alignas(16) float fin[2][kHG];     // of a stretch: factors of the output,
    alignas(16) float flush[2][kHG];   // and of the partial so far
    WorkSmem work;
};

// 2 x 16 lanes of tensor memory: threads 0..15 read lanes 0..15 of the address at
// columns c .. c + 15, threads 16..31 the same lanes at columns c + 16 .. c + 31.
__device__ __forceinline__ void tmem_ld16x2_next_raw(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16], 16;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the nearest e5m2 values of two f16, the first in the low byte
__device__ __forceinline__ uint32_t f16x2_e5m2x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

// The next term of four f16 numbers (two words): their upper bytes, which are
// e5m2 values; the numbers keep the rest.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t &a, uint32_t &b) {
    const uint32_t t = __byte_perm(a, b, 0x7531);
    a = f16x2_sub(a, a & 0xFF00FF00u);
    b = f16x2_sub(b, b & 0xFF00FF00u);
    return t;
}
__device__ __forceinline__ uint32_t last_bytes(uint32_t a, uint32_t b) {
    return f16x2_e5m2x2(a) | f16x2_e5m2x2(b) << 16;
}

// Four weights as kTerms words of four e5m2 values each.
template <int kTerms>
__device__ __forceinline__ void split_weights(const float (&p)[4], uint32_t (&t)[kTerms]) {
    uint32_t a = f16x2(p[0], p[1]), b = f16x2(p[2], p[3]);
    if constexpr (kTerms == 3) {
        t[0] = upper_bytes(a, b);
        t[1] = upper_bytes(a, b);
        t[2] = last_bytes(a, b);
    } else {
        // four terms hold f16's 11 bits (but for what is below e5m2's last place),
        // the rest of the f32 number makes two more
        uint32_t ra = a, rb = b;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = upper_bytes(ra, rb);
        const float2 ha = f16x2_values(f16x2_sub(a, ra)), hb = f16x2_values(f16x2_sub(b, rb));
        a = f16x2(p[0] - ha.x, p[1] - ha.y);
        b = f16x2(p[2] - hb.x, p[3] - hb.y);
        t[4] = upper_bytes(a, b);
        t[5] = last_bytes(a, b);
    }
}

// One head of the query as the operand's rows r (hi) and r + 16 (lo) of 128; a
// lane has 16 columns.  Returns the factor that takes sums of codes back to the
// query's units (NaN where the query is not finite).
__device__ __forceinline__ float split_query(const uint4 (&raw)[2], uint8_t *sQ, int r, int lane) {
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    // 1.m 2^(e - 127) to 2^7
    const int k = min(134 - static_cast<int>(top >> 7), 126);
    const float f = exponent_f32(k);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[2 * j] = __uint_as_float(w[2 * i + j] << 16) * f;
            x[2 * j + 1] = __uint_as_float(w[2 * i + j] & 0xFFFF0000u) * f;
        }
        hi[i] = e4m3x4(x[0], x[1], x[2], x[3]);
        float h[4];
        e4m3x4_values(hi[i], h);
        lo[i] = e4m3x4(x[0] - h[0], x[1] - h[1], x[2] - h[2], x[3] - h[3]);
    }
    uint8_t *const at = sQ + (lane >> 3) * (2 * kHG * 128) + (r >> 3) * 1024 + (r & 7) * 128 +
                        (((lane & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(at + 2 * 1024) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    return top >= 0x7F80u ? NAN : exponent_f32(-k);
}

// kTerms: e5m2 terms of P (6 for an f32 output, 3 for bf16).
template <int kTerms>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_fp8_kernel(const __grid_constant__ CUtensorMap tm_rows, const PagedFp8Args A) {
    constexpr bool kBf16 = kTerms == 3;
    constexpr int kFlush = kBf16 ? kFlushBf16 : kFlushF32;
    constexpr int kPiece = kPieceBytes<kTerms>;          // 16 rows of P
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem<1024>(smem_raw);
    uint8_t *sQ = smem;                                  // [4 col groups][128 rows][128 B]
    uint8_t *sRows = sQ + kQBytes;                       // [stage][8 groups][4 col groups][8 rows][128 B]
    uint8_t *sP = sRows + kStages * kStageBytes;         // [16 rows of the chunk][term][64 heads][16 B]
    uint8_t *sOut = sP + kChunk / 16 * kPiece;           // [epilogue warp][16 heads][32 columns], bf16 output
    Smem &S = *reinterpret_cast<Smem *>(sOut + kStagedBytes<kTerms>);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = blockIdx.y, h0 = hg * kHG;
    const int H = A.H;

    if (tid == 0) {
        mbar_init(&S.q_full, kSmThreads);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&S.full[i], kSlices);
            for (int k = 0; k < kSteps; ++k) mbar_init(&S.empty[i][k], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.sfree[i], kSmThreads);
            mbar_init(&S.pfull[i], kSmThreads);
            mbar_init(&S.stretch[i], kSmThreads);
            mbar_init(&S.stretch_free[i], kSmThreads);
        }
        mbar_init(&S.pfree, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&S.ofree[i], kSmThreads);
        mbar_fence_init();
        tma_prefetch_desc(&tm_rows);
    }
    if (warp == 8) {
        tmem_alloc(&S.tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    Work<kChunk, kSegCost, kCutAbove> W(A, S.work);
    W.count();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_holder;
    W.divide();
    W.first_list();
    const int ndt = W.ndt, dt0 = W.dt0;                  // 128-column tiles of this CTA
    const Rec *const rec = S.work.rec;

    // pipeline positions, kept across lists of segments
    uint32_t n_fetch = 0;                // chunks fetched
    uint32_t nq = 0, np = 0;             // chunks whose S / O^T product was issued
    uint32_t n_ql = 0;                   // queries used
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
            // all four drain O^T where that chunk ends a stretch.
            constexpr uint32_t id_qk = idesc_fp8<2 * kHG, kChunk, false, false>();
            constexpr uint32_t id_pv = idesc_fp8<128, kHG, true, true>(), id_wide = idesc_fp8<128, 2 * kHG, true, true>();
            const uint64_t q_desc = sw128_desc(smem_addr(sQ), 16, 1024);
            const uint64_t r_desc = sw128_desc(smem_addr(sRows), 16, kGroupBytes);
            const uint64_t a_desc = sw128_desc(smem_addr(sRows) + dt0 * 1024, 1024, kGroupBytes);
            const uint64_t p_desc = atom_desc(smem_addr(sP), kPiece, 128);
            const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int hmax = min(kHG, H - h0);
            auto product = [&](int dd, int ks, uint64_t ad, uint32_t acc) {
                const uint64_t av = ad + off(dd * 1024 + ks * 4 * kGroupBytes);
                const uint32_t d = tmem + o_col(dd);
                const uint64_t pd = p_desc + off(2 * ks * kPiece);
                if (dd < kWide) {
#pragma unroll
                    for (int t = 0; t + 1 < kTerms; t += 2)
                        umma_fp8(d, av, pd + off(t * kTermBytes), id_wide, t > 0 ? 1u : acc);
                    if (kTerms & 1) umma_fp8(d, av, pd + off((kTerms - 1) * kTermBytes), id_pv, 1u);
                } else {
#pragma unroll
                    for (int t = 0; t < kTerms; ++t)
                        umma_fp8(d, av, pd + off(t * kTermBytes), id_pv, t > 0 ? 1u : acc);
                }
            };
            auto pv = [&](auto ntile, uint64_t ad, int st, int ks) {
#pragma unroll
                for (int dd = 0; dd < ntile; ++dd) product(dd, ks, ad, 1u);
                umma_commit(&S.empty[st][ks]);
                if (ks + 1 == kSteps) umma_commit(&S.pfree);
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
                        for (int kk = 0; kk < kHD / 32; ++kk) {
                            const uint32_t cg = kk >> 2, ko = (kk & 3) * 32;
                            umma_fp8(d, q_desc + off(cg * (2 * kHG * 128) + ko), rd + off(cg * 1024 + ko), id_qk,
                                     kk > 0 ? 1u : 0u);
                        }
                        umma_commit(&S.sfull[sb]);
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
                                for (int ks = 0; ks < kSteps; ++ks) product(dd, ks, ad, ks > 0 ? 1u : 0u);
                                if (dd + 1 == ndt) {
                                    for (int ks = 0; ks < kSteps; ++ks) umma_commit(&S.empty[st][ks]);
                                    umma_commit(&S.pfree);
                                }
                            }
                            __syncwarp();
                        }
                    } else {
#pragma unroll
                        for (int ks = 0; ks < kSteps; ++ks) {
                            if (ks > 0) mbar_wait(&S.pfull[ks], pp, A.status);
                            __syncwarp();
                            tc_fence_after();
                            if (elect_one()) {
                                if (ndt == 4) pv(std::integral_constant<int, 4>{}, ad, st, ks);
                                else if (ndt == 2) pv(std::integral_constant<int, 2>{}, ad, st, ks);
                                else pv(std::integral_constant<int, 1>{}, ad, st, ks);
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
                        drain_stretch<kBf16, kWide>(A, tmem + lane_off + kOCol, S.fin[e], S.flush[e], S.ofree, sOut, dt0,
                                                    ndt, hmax, obase, pslot, add, part);
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
            // number is on its way from the table, two before it its scale.
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
                int32_t page, at;                      // row of the page; or (page -2) of the rings; < 0: no row
                bool box;                              // 8 rows of one page from here on
            };
            auto look_up = [&](const Cursor &k) {
                Entry e{-1, -1, false};
                if (k.i >= nrec) return e;
                const Rec &r = rec[k.i];
                const int j = k.c * kChunk + 16 * li + rl, w = j - rec_window_slot(r);
                if (j < r.n) {
                    const int pg = static_cast<int>(A.page_div.div(j));
                    e.at = j - pg * A.L.page_rows;
                    e.page = A.L.table[static_cast<int64_t>(r.b) * A.L.max_pages + pg];
                    e.box = j + 8 <= r.n && e.at + 8 <= A.L.page_rows;
                    if (e.page == -2) e.page = -1;
                } else if (w >= 0 && w < r.near) {
                    const int64_t x = r.first + w;
                    e.page = -2;
                    if (x < r.first_res) bad |= CSA_DEV_MISSING_SWA;
                    else e.at = r.b * A.L.swa_cap + static_cast<int32_t>(A.swa_div.mod64(x));
                }
                return e;
            };
            struct Place {
                const uint8_t *src;                    // the row's codes, or null
                float scale;
                int32_t row;                           // row of the pool, or -1
                uint32_t box;                          // bit g: group g of 8 rows is one box
            };
            auto place = [&](const Entry &e) {
                Place p{nullptr, 0.f, -1, 0};
                if (e.at >= 0) {
                    if (e.page == -2) {
                        p.src = static_cast<const uint8_t *>(A.L.swa_kv) + static_cast<int64_t>(e.at) * kHD;
                        p.scale = __ldcg(A.swa_scales + e.at);
                    } else if (e.page < 0 || e.page >= A.num_pages) {
                        bad |= CSA_DEV_BAD_INDEX;
                    } else {
                        p.row = static_cast<int32_t>(e.page * A.page_stride) + e.at;
                        if (!CSA_CHECK(p.row < A.total_rows, A.status)) {
                            p.row = -1;
                        } else {
                            p.src = A.codes + static_cast<int64_t>(p.row) * kHD;
                            p.scale = __ldcg(A.scales + e.page * A.scale_stride + e.at);
                        }
                    }
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
                const uint32_t okm = __ballot_sync(0xffffffffu, now.src != nullptr) & 0xFFFFu;
                const int32_t y1 = __shfl_sync(0xffffffffu, now.row, 8);
                const int st = n_fetch % kStages;
                const uint32_t ph = ((n_fetch / kStages) & 1u) ^ 1u;
                uint64_t *const empty = &S.empty[st][li / 2];
                if (pending >= 0 && !__all_sync(0xffffffffu, mbar_test_wait(empty, ph))) land(false);
                mbar_wait(empty, ph, A.status);
                __syncwarp();
                uint8_t *rows = sRows + st * kStageBytes + 2 * li * kGroupBytes;
                if (lane < 16) {
                    S.scale[st][16 * li + rl] = now.scale;
                    S.scale_log[st][16 * li + rl] =
                        now.src ? __log2f(fminf(fmaxf(fabsf(now.scale), 0x1p-60f), 0x1p60f)) : 0.f;
                }
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
                            const uint8_t *p = reinterpret_cast<const uint8_t *>(__shfl_sync(
                                0xffffffffu, reinterpret_cast<unsigned long long>(now.src), 8 * g + rr));
                            cp_async16(rows + g * kGroupBytes + (lane >> 3) * 1024 + rr * 128 + (((lane & 7) ^ rr) << 4),
                                       p ? p + lane * 16 : A.codes, p != nullptr);
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
                if (by_row) {
                    pending = st;
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.full[st]);
                }
                ++n_fetch;
            }
            if (pending >= 0) land(false);
            bad = static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad)));
            if (lane == 0 && W.lead) raise_status(A.status, bad);
        } else if (warp >= 4 && warp < 8) {
            // -------------------------------------------- the query, softmax
            const int q = warp & 3;                  // TMEM lane quarter
            const int hl = q * 16 + (lane & 15);     // head of this lane (two lanes per head)
            const bool upper = lane >= 16;           // rows 16..31 and 48..63 of the chunk, others 0..15 and 32..47
            const bool hv = h0 + hl < H;
            const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
            for (int i = 0; i < nrec; ++i) {
                const int nch = rec[i].c1 - rec[i].c0;
                if (nch <= 0) {
                    if (rec[i].flags & kRecZero) {
                        const int64_t obase = (static_cast<int64_t>(rec[i].t) * H + h0) * kHD;
                        for (int x = tid - 128; x < min(kHG, H - h0) * 128 * ndt; x += kSmThreads) {
                            const int64_t at = obase + (x / (128 * ndt)) * kHD + dt0 * 128 + x % (128 * ndt);
                            if (kBf16) static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(0.f);
                            else static_cast<float *>(A.out)[at] = 0.f;
                        }
                    }
                    continue;
                }
                // (the segment before this one is done with Q: its last logits have
                // come)  Four heads' loads at a time.
                float c = 0.f;
                const uint4 *const src = reinterpret_cast<const uint4 *>(
                    A.q + (static_cast<int64_t>(rec[i].t) * H + h0 + q * 16) * kHD) + 2 * lane;
#pragma unroll 1
                for (int g = 0; g < 16; g += 4) {
                    uint4 raw[4][2];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            raw[x][y] = h0 + q * 16 + g + x < H ? __ldcg(src + (g + x) * (kHD / 8) + y) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float f = split_query(raw[x], sQ, 32 * q + g + x, lane);
                        if ((lane & 15) == g + x) c = f * A.scale_log2;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&S.q_full);

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
                    float x[32];
                    {
                        uint32_t hi[2][16], lo[2][16];
                        const uint32_t at = tmem + lane_off + kSCol + sb * 64;
                        tmem_ld16x2_next_raw(at, hi[0]);
                        tmem_ld16x2_next_raw(at + (16u << 16), lo[0]);
                        tmem_ld16x2_next_raw(at + 32, hi[1]);
                        tmem_ld16x2_next_raw(at + (16u << 16) + 32, lo[1]);
                        tmem_wait_ld();
                        tc_fence_before();
                        mbar_arrive(&S.sfree[sb]);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            x[j] = __uint_as_float(hi[j >> 4][j & 15]) + __uint_as_float(lo[j >> 4][j & 15]);
                    }
                    mbar_wait(&S.full[st], (n_sm / kStages) & 1u, A.status);   // orders masks and scales
                    const uint32_t m0 = S.maskw[st][upper ? 1 : 0], m1 = S.maskw[st][upper ? 3 : 2];
                    const bool all = __all_sync(0xffffffffu, (m0 & m1) == 0xFFFFu);
                    // logits; the maximum is that of the logits plus their scales' logarithms
                    const float *const sc = S.scale[st] + (upper ? 16 : 0), *const sl = S.scale_log[st] + (upper ? 16 : 0);
                    float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const int at = (j & 15) + (j >> 4) * 32;
                        const float4 s4 = *reinterpret_cast<const float4 *>(sc + at);
                        const float4 l4 = *reinterpret_cast<const float4 *>(sl + at);
                        const float s[4] = {s4.x, s4.y, s4.z, s4.w}, lg[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[j + e] *= s[e] * c;
                        if (!all) {
                            const uint32_t m = j < 16 ? m0 : m1;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!(m >> ((j & 15) + e) & 1u)) x[j + e] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) mq[e] = fmaxf(mq[e], x[j + e] + lg[e]);
                    }
                    float mc = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
                    mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 16));
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
                        for (int y = 0; y < static_cast<int>(o_col(ndt) - kOCol); y += 16) {
                            uint32_t o[16];
                            const uint32_t ta2 = tmem + lane_off + kOCol + y;
                            tmem_ld16_raw(ta2, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * S.alpha[y % kHG + e]);
                            tmem_st16(ta2, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        named_bar_sync(kBarSm, kSmThreads);
                    }
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref - kTop;
                    float sq[2] = {0.f, 0.f};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[4][kTerms];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 s4 = *reinterpret_cast<const float4 *>(sc + half * 32 + 4 * u);
                            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
                            float p[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                p[e] = fast_exp2(x[half * 16 + 4 * u + e] - mr);
                                sq[e & 1] += p[e];
                                p[e] *= s[e];
                            }
                            split_weights<kTerms>(p, w[u]);
                        }
                        if (half == 0 && n_sm > 0) mbar_wait(&S.pfree, (n_sm - 1) & 1u, A.status);
                        uint8_t *const at = sP + (2 * half + (upper ? 1 : 0)) * kPiece + hl * 16;
#pragma unroll
                        for (int t = 0; t < kTerms; ++t)
                            *reinterpret_cast<uint4 *>(at + t * kTermBytes) = make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]);
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
                            if (A.sinks && hv) zs += exp2f(A.sinks[h0 + hl] * kLog2e - mr);
                            f = m_ref == -INFINITY && l == 0.f ? 0.f : 1.f / zs;     // (a sink of NaN: NaN)
                        }
                        S.fin[e][hl] = f;
                        if (last && cut && dt0 == 0)
                            A.part_ml[(static_cast<int64_t>(rec[i].slot) * gridDim.y + hg) * kHG + hl] =
                                make_float2(m_ref == -INFINITY ? m_ref : mr, l);
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
size_t smem_bytes() {
    return 1024 + kQBytes + kStages * kStageBytes + kChunk / 16 * kPieceBytes<kTerms> + kStagedBytes<kTerms> + sizeof(Smem);
}

constexpr size_t kSmemMost = 227 * 1024;
static_assert(1024 + kQBytes + kStages * kStageBytes + kChunk / 16 * kPieceBytes<6> + kStagedBytes<6> + sizeof(Smem) <= kSmemMost);
static_assert(1024 + kQBytes + kStages * kStageBytes + kChunk / 16 * kPieceBytes<3> + kStagedBytes<3> + sizeof(Smem) <= kSmemMost);

}  // namespace

cudaError_t launch_paged_attention_fp8(const Launch &lc, const csa_paged_layout_t &L,
                                       const csa_params_t &p, const void *cache, const float *scales,
                                       const float *swa_scales, int64_t num_pages,
                                       int64_t page_stride, int64_t scale_stride, const void *q,
                                       const float *sinks, csa_type_t out_type, void *out,
                                       int32_t *status, void *ws) {
    CUtensorMap tr;
    {
        // [128 columns][rows of the pool][4 column groups]
        const uint64_t dims[3] = {128, static_cast<uint64_t>(paged_rows(L, num_pages, page_stride)), 4};
        const uint64_t strides[2] = {kHD, 128};
        const uint32_t box[3] = {128, 8, 4};
        if (encode_tensor_map_u8(&tr, cache, 3, dims, strides, box) != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    PagedFp8Args A{};
    static_cast<PagedArgs &>(A) = paged_args(lc, L, p, num_pages, page_stride, sinks, out_type, out, status, ws);
    A.codes = static_cast<const uint8_t *>(cache);
    A.scales = scales;
    A.swa_scales = swa_scales;
    A.scale_stride = scale_stride;
    A.q = static_cast<const __nv_bfloat16 *>(q);
    const int groups = groups_of(p), ctas = static_cast<int>(A.split_div[0].d);
    auto launch = [&](auto terms) {
        constexpr int kTerms = decltype(terms)::value;
        constexpr auto kernel = paged_attention_fp8_kernel<kTerms>;
        const cudaError_t e = prepare_kernel<kernel>(smem_bytes<kTerms>());
        return e != cudaSuccess ? e : launch_pdl(kernel, dim3(ctas, groups), dim3(kThreads), smem_bytes<kTerms>(), lc.stream, tr, A);
    };
    const cudaError_t e = A.bf16_out ? launch(std::integral_constant<int, 3>{}) : launch(std::integral_constant<int, 6>{});
    if (e != cudaSuccess) return e;
    // no token can be cut: nothing to join
    const int64_t slots_max = (static_cast<int64_t>(L.max_pages) * L.page_rows + 7) / 8 * 8 + p.window;
    if (slots_max <= kCutAbove * kChunk) return cudaSuccess;
    const int entries = L.num_tokens < ctas ? L.num_tokens : ctas;
    // one long context is cut into many parts, a batch's tokens into few
    const PagedArgs &B = A;
    return A.bf16_out ? launch_join<true>(lc, B, entries, groups, slots_max)
                      : launch_join<false>(lc, B, entries, groups, slots_max);
}

}  // namespace csa
