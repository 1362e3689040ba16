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

#include "csa_device.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kSmThreads = 128;                 // warps 4..7; the epilogue's 8..11
constexpr int kBarSm = 1;
constexpr int kHG = 64;                         // heads per CTA
constexpr int kChunk = 48;
constexpr int kSlices = kChunk / 16;            // of 16 rows: one K step of O^T each
constexpr int kQBytes = kHG * kHD * 2;          // 64 KiB
constexpr int kGroupBytes = 8 * kHD * 2;        // 8 rows: 8 KiB
constexpr int kStageBytes = kChunk / 8 * kGroupBytes;   // 48 KiB
constexpr int kStages = 3;
constexpr int kPBytes = kHG * kChunk * 2;       // one bf16 term of P: 6 KiB
constexpr int kOutBytes = 1024;                 // of an epilogue warp: 32 columns x 16 heads in bf16
template <int kTerms>
constexpr int kStagedBytes = kTerms == 1 ? 4 * kOutBytes : 0;
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
constexpr int kMaxCtas = 152;                   // CTAs of the grid at most (sizes the workspace)
constexpr int kSegCost = 4;                     // a segment's epilogue, in chunks (3: 128 contexts of 512 rows 30.3
                                                // us instead of 29.3; 2: 128-head drafts 82.5 instead of 76.5)
constexpr int kCutAbove = 5;                    // chunks a token may exceed the mean before tokens are cut
constexpr int kFlushF32 = 53, kFlushBf16 = 682; // chunks between roundings of the accumulator, at most

struct PagedArgs {
    csa_paged_layout_t L;
    int32_t H, window, ratio, bf16_out;
    float scale_log2;
    int32_t total_rows;       // rows of the pool: the coordinate that reads as zeros
    FastDiv page_div, ratio_div, swa_div;   // by page_rows, ratio, swa_cap
    FastDiv split_div[3];
    int64_t num_pages, page_stride;
    const __nv_bfloat16 *cache;
    const float *sinks;
    void *out;
    float4 *part_o;           // [slot][head group][tile][16 quads of heads][128 columns]: 4 heads
    float2 *part_ml;          // [slot][head group][64 heads]: m (log2 units), l
    int2 *meta;               // by token (T <= CTAs) or by CTA: first slot, parts (0: none)
    int32_t *status;
};

// One segment: chunks [c0, c1) of token t.
struct Rec {
    int32_t t, b;             // b < 0: padding
    int32_t n, near;          // compressed rows, window rows
    int32_t c0, c1;
    int32_t slot;             // partial slot
    int32_t flags;
    int64_t first;            // first window position
    int64_t first_res;        // oldest position the ring holds
};
constexpr int kRecPart = 1;   // part of a cut token: leaves (O, m, l)
constexpr int kRecZero = 2;   // a token without rows: zeros

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
    int32_t nrec, more;
    int32_t t0, s0;
    int2 wsum[kThreads / 32];    // cost, most chunks of a token
    Rec rec[kMaxRec];
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, int32_t x, int32_t y,
                                            int32_t z, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

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

// Unswizzled K-major operand: atoms of 8 rows x 16 bytes, 128 contiguous bytes
// each, `lbo` apart along K and `sbo` along the rows.
__device__ __forceinline__ uint64_t atom_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return sw128_desc(saddr, lbo, sbo) & ~(static_cast<uint64_t>(7u) << 61);
}

// a byte offset as a step of a descriptor's start-address field (every shared
// address is below 256 KiB, so the field never carries)
__device__ __forceinline__ constexpr uint64_t off(uint32_t bytes) { return bytes >> 4; }

// What token t attends: b < 0 for padding, n = near = 0 for a bad token.
// `per` tokens a sequence is the guess by which the sequence's length is
// loaded in the same round trip as its number.
__device__ __forceinline__ Rec token_rec(const PagedArgs &A, int t, int per, int &bad) {
    Rec r{};
    r.t = t;
    const int g = min(t / per, A.L.num_seqs - 1);
    r.b = __ldcg(A.L.tok_seq + t);
    const int64_t pos = __ldcg(A.L.tok_pos + t);
    int64_t n = __ldcg(A.L.row_len + g);
    if (A.window > 0) r.first_res = __ldcg(A.L.swa_first_pos + g);
    bad = 0;
    if (r.b == -1) return r;
    if (r.b < 0 || r.b >= A.L.num_seqs || pos < 0) {
        bad = CSA_DEV_BAD_LAYOUT;
        r.b = 0;
        return r;
    }
    if (r.b != g) {
        n = __ldcg(A.L.row_len + r.b);
        if (A.window > 0) r.first_res = __ldcg(A.L.swa_first_pos + r.b);
    }
    const int64_t cap = static_cast<int64_t>(A.L.max_pages) * A.L.page_rows;
    if (n < 0) {
        bad |= CSA_DEV_BAD_LENGTH;
        n = 0;
    }
    if (n > cap) {
        bad |= CSA_DEV_CAPACITY;
        n = cap;
    }
    const int64_t seen = A.ratio_div.div64(pos);
    r.n = static_cast<int32_t>(n < seen ? n : seen);
    if (A.window > 0) {
        r.first = window_first(pos, A.window);
        r.near = static_cast<int32_t>(pos - r.first + 1);
    }
    return r;
}

__device__ __forceinline__ int rec_window_slot(const Rec &r) { return (r.n + 7) & ~7; }
__device__ __forceinline__ int rec_slots(const Rec &r) {
    return r.near > 0 ? rec_window_slot(r) + r.near : r.n;
}
__device__ __forceinline__ int rec_chunks(const Rec &r) {
    return r.b < 0 ? 0 : (rec_slots(r) + kChunk - 1) / kChunk;
}
__device__ __forceinline__ int chunk_cost(int chunks) { return chunks > 0 ? chunks + kSegCost : 1; }

// Chunks after which a segment of nch chunks rounds its accumulator into the
// partial: equal stretches of at most kMost.
template <int kMost>
__device__ __forceinline__ int flush_every(int nch) {
    const int n = (nch + kMost - 1) / kMost;
    return n > 1 ? (nch + n - 1) / n : nch;
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
    const int G = gridDim.x, hg = blockIdx.y, h0 = hg * kHG;
    const int T = A.L.num_tokens, H = A.H;

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
            mbar_init(&S.stretch_free[i], kSmThreads);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&S.ofree[i], kSmThreads);
        mbar_fence_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_rows);
    }
    if (warp == 8) {
        tmem_alloc(&S.tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();

    // ---------------------------------------------------- division of the work
    // (the layout is read before the wait for the preceding kernel, as
    // everywhere in this library)  Chunks and costs of all tokens, a
    // contiguous run of tokens per thread; with one token a thread its record
    // stays in registers.
    const int tps = max(1, T / A.L.num_seqs);
    const int per = (T + kThreads - 1) / kThreads;
    const int ta = min(T, tid * per), te = min(T, ta + per);
    Rec own{};
    int own_c = 0, own_bad = 0;
    int cost = 0, maxc = 0;
    for (int t = ta; t < te; ++t) {
        own = token_rec(A, t, tps, own_bad);
        own_c = rec_chunks(own);
        cost += chunk_cost(own_c);
        maxc = max(maxc, own_c);
    }
    int incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    maxc = __reduce_max_sync(0xffffffffu, maxc);
    if (lane == 31) S.wsum[warp] = make_int2(incl, maxc);
    if (tid == 0) {
        S.t0 = T;
        S.nrec = 0;
        S.more = 0;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_holder;
    int base = 0, U = 0;                 // units in front of this warp, of all tokens
    maxc = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) base = U;
        U += S.wsum[w].x;
        maxc = max(maxc, S.wsum[w].y);
    }
    // Tokens are cut only where that shortens the longest CTA by more than
    // the partials and their join cost: otherwise CTA c takes token c (T <= G),
    // or the tokens that begin in its range.  (240 rows; 2 and 3 chunks measure
    // the same within 0.5%.  At 8 chunks 64 tokens of 512 rows gain, 27.6 -> 26.4
    // us, and one of 256 rows loses, 9.4 -> 15.4.  At 16, 150 tokens of 250 to 500
    // rows gain, 30.8 -> 26.6 us, and 64 of 512 rows, 27.6 -> 23.4, but 64 of 512
    // to 1,024 rows lose, 27.9 -> 34.3, 128 of 32 to 1,024 rows, 31.4 -> 46.3, and
    // one of 600, 9.0 -> 22.8.)
    const bool direct = T <= G && maxc <= static_cast<int>(A.split_div[0].div(U)) + kCutAbove;
    const bool snap = direct || (T > G && maxc <= kCutAbove);
    // few CTAs at work: 2 or 4 of them share a range, each with all of its
    // logits and weights and its share of the 512 columns: the last products
    // and the partial (32 bytes a cycle and SM) are that much shorter (8,192
    // rows, three chunks for two CTAs 14.8 us, two for one 15.3)
    int dlog = 0;
    if (direct) dlog = T * 4 <= G ? 2 : T * 2 <= G ? 1 : 0;
    else if (!snap && T <= G) dlog = U <= G / 4 ? 2 : U <= G + G / 3 ? 1 : 0;
    const int dparts = 1 << dlog;
    const int split = static_cast<int>(blockIdx.x) >> dlog;
    const int ndt = 4 >> dlog;                                    // 128-column tiles of this CTA
    const int dt0 = (static_cast<int>(blockIdx.x) & (dparts - 1)) * ndt;
    // equal ranges of `share` units, the last ones shorter or empty: as few parts
    // as the longest range allows
    const int share = static_cast<int>(A.split_div[dlog].div(U + (G >> dlog) - 1));
    int ua = 0, ub = split < T ? 1 : 0;
    if (!direct) {
        ua = min(split * share, U);
        ub = min(ua + share, U);
    }
    const bool by_token = T <= G;
    const bool lead = hg == 0 && dt0 == 0;       // reports errors, writes the join's list
    // The first token of the range: the one that holds unit ua, or (whole
    // tokens only) the first that begins at or behind it.
    if (direct) {
        if (tid == 0) S.t0 = split;
    } else {
        int s = base + incl - cost;
        for (int t = ta; t < te; ++t) {
            int bad;
            const int c = per == 1 ? own_c : rec_chunks(token_rec(A, t, tps, bad));
            const int e = s + chunk_cost(c);
            if (snap ? s >= ua : (s <= ua && ua < e)) {
                if (snap) {
                    atomicMin(&S.t0, t);
                } else {
                    S.t0 = t;
                    S.s0 = s;
                }
                break;
            }
            s = e;
        }
    }
    __syncthreads();
    if (per > 1 && snap && !direct) {
        int s = base + incl - cost;
        for (int t = ta; t < te; ++t) {
            if (t == S.t0) S.s0 = s;
            int bad;
            s += chunk_cost(rec_chunks(token_rec(A, t, tps, bad)));
        }
        __syncthreads();
    }
    int t0 = S.t0, s0 = S.s0;

    // Lists the segment of one token (whose units begin at s) as entry `at`.
    // Returns the token's entry for the join; `owner`: its first chunk is here.
    auto list = [&](Rec &r, int c, int s, int at, bool &owner) {
        int2 m = make_int2(-1, 0);
        owner = true;
        r.c0 = 0;
        r.c1 = c;
        r.slot = 2 * split + 1;
        if (!snap) {
            owner = s >= ua;
            r.c0 = min(max(ua - s, 0), c);
            r.c1 = min(ub - s, c);
            if (!owner) r.slot = 2 * split;
            // the split that holds the token's last chunk
            if (owner && c > 0) {
                const int last = (s + c - 1) / share;
                if (last > split) m = make_int2(r.slot, last - split + 1);
            }
            if (r.c1 - r.c0 < c) r.flags |= kRecPart;
        }
        if (r.b >= 0 && c == 0 && owner) r.flags |= kRecZero;
        S.rec[at] = r;
        atomicAdd(&S.nrec, 1);
        // its first table entry on its way while the roles start
        if (r.c0 * kChunk < r.n)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(A.L.table + static_cast<int64_t>(r.b) * A.L.max_pages +
                                                          A.page_div.div(r.c0 * kChunk)));
        if (at == kMaxRec - 1 && !direct) {
            S.more = 1;
            S.s0 = s + chunk_cost(c);
        }
        return m;
    };
    auto report = [&](const Rec &r, int bad, int2 m) {
        raise_status(A.status, bad);
        if (by_token) {
            A.meta[r.t] = m;
        } else if (m.y > 0) {
            A.meta[split] = m;
            A.meta[G + split] = make_int2(r.t, 0);
        }
    };
    // thread i lists token t0 + i
    auto list_next = [&]() {
        Rec r{};
        int bad = 0, c = 0, w = 0;
        const bool in = tid < kMaxRec && t0 + tid < T && ub > ua;
        if (in) {
            r = token_rec(A, t0 + tid, tps, bad);
            c = rec_chunks(r);
            w = chunk_cost(c);
        }
        int run = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += v;
        }
        if (lane == 31) S.wsum[warp].x = run;
        __syncthreads();
        int s = s0 + run - w;
        for (int k = 0; k < kMaxRec / 32; ++k)
            if (k < warp) s += S.wsum[k].x;
        if (in && s < ub) {
            bool owner;
            const int2 m = list(r, c, s, tid, owner);
            if (lead && owner) report(r, bad, m);
        }
    };
    if (per == 1) {
        // the first list, from the registers
        const int at = tid - t0;
        const int s = base + incl - cost;
        bool owner = false;
        int2 m = make_int2(-1, 0);
        if (at >= 0 && at < kMaxRec && tid < T && ub > ua && (direct ? at == 0 : s < ub))
            m = list(own, own_c, s, at, owner);
        pdl_wait();
        pdl_launch_dependents();
        if (!by_token) {
            if (lead && tid == 0) A.meta[split] = make_int2(-1, 0);
            __syncthreads();
        }
        if (lead && owner) report(own, own_bad, m);
    } else {
        pdl_wait();
        pdl_launch_dependents();
        if (lead && tid == 0) A.meta[split] = make_int2(-1, 0);
        list_next();
    }

    // pipeline positions, kept across lists of segments
    uint32_t n_fetch = 0;                // chunks fetched
    uint32_t nq = 0, np = 0;             // chunks whose S / O^T product was issued
    uint32_t n_ql = 0;                   // Q loads issued
    uint32_t n_sm = 0;                   // chunks through the softmax; whose O^T product was issued
    uint32_t n_ep = 0;                   // stretches through the softmax, the epilogue

    for (;;) {
        __syncthreads();
        t0 += kMaxRec;
        s0 = S.s0;
        const int nrec = S.nrec;
        const bool more = S.more != 0;
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
            const int dl = (warp & 3) * 32 + lane;   // column of a tile
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
                    nch = S.rec[i].c1 - S.rec[i].c0;
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
                            tma_load_4d(sQ, &tm_q, 0, h0, 0, S.rec[i].t, &S.q_full, policy_evict_normal());
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
                        const int t = S.rec[bi].t, flags = S.rec[bi].flags;
                        const int64_t obase = (static_cast<int64_t>(t) * H + h0) * kHD;
                        const int64_t pslot = static_cast<int64_t>(S.rec[bi].slot) * gridDim.y + hg;
                        const int e = n_ep & 1u;
                        (void)CSA_CHECK(S.rec[bi].slot < 2 * G && t < T, A.status);
                        const bool add = bk >= be;               // the partial holds earlier stretches
                        const bool part = (flags & kRecPart) || bk + 1 < bn;
                        mbar_wait(&S.stretch[e], (n_ep >> 1) & 1u, A.status);
                        mbar_wait(&S.pfree, (n_sm - 1) & 1u, A.status);   // its last product
                        ++n_ep;
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int dd = 0; dd < ndt; ++dd) {
                            // one column per lane; a partial keeps four heads together,
                            // so that a warp stores 512 contiguous bytes
                            float4 *const pd = A.part_o + (pslot * 4 + dt0 + dd) * (16 * 128) + dl;
#pragma unroll 1
                            for (int hb = 0; hb < kHG; hb += 32) {
                                if (hb >= hmax) break;
                                uint32_t o[32];
                                const uint32_t oc = tmem + lane_off + o_col<kTerms>(dd) + hb;
                                tmem_ld16_raw(oc, *reinterpret_cast<uint32_t(*)[16]>(o));
                                tmem_ld16_raw(oc + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
                                float4 *const pq = pd + hb / 4 * 128;
                                if (dd < kWide<kTerms>) {
#pragma unroll
                                    for (int y = 0; y < 32; y += 16) {
                                        uint32_t lo[16];
                                        tmem_ld16_raw(oc + kHG + y, lo);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int x = 0; x < 16; ++x)
                                            o[x + y] = __float_as_uint(__uint_as_float(o[x + y]) + __uint_as_float(lo[x]));
                                    }
                                }
                                if (add) {
                                    float4 old[8];
#pragma unroll
                                    for (int x = 0; x < 8; ++x) old[x] = pq[x * 128];
                                    tmem_wait_ld();
#pragma unroll
                                    for (int x = 0; x < 8; ++x) {
                                        const float4 f = *reinterpret_cast<const float4 *>(S.flush[e] + hb + 4 * x);
                                        o[4 * x] = __float_as_uint(fmaf(old[x].x, f.x, __uint_as_float(o[4 * x])));
                                        o[4 * x + 1] = __float_as_uint(fmaf(old[x].y, f.y, __uint_as_float(o[4 * x + 1])));
                                        o[4 * x + 2] = __float_as_uint(fmaf(old[x].z, f.z, __uint_as_float(o[4 * x + 2])));
                                        o[4 * x + 3] = __float_as_uint(fmaf(old[x].w, f.w, __uint_as_float(o[4 * x + 3])));
                                    }
                                }
                                tmem_wait_ld();
                                if (hb + 32 >= hmax) {           // the tile is in registers
                                    tc_fence_before();
                                    mbar_arrive(&S.ofree[dd]);
                                }
                                if (part) {
#pragma unroll
                                    for (int x = 0; x < 8; ++x)
                                        pq[x * 128] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                                                  __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
                                    continue;
                                }
                                // (all factors before the first store, which the compiler
                                // would not let a later factor's load pass: 5,600 instead
                                // of 14,100 cycles for 64 heads)
#pragma unroll
                                for (int x = 0; x < 8; ++x) {
                                    const float4 f = *reinterpret_cast<const float4 *>(S.fin[e] + hb + 4 * x);
                                    o[4 * x] = __float_as_uint(__uint_as_float(o[4 * x]) * f.x);
                                    o[4 * x + 1] = __float_as_uint(__uint_as_float(o[4 * x + 1]) * f.y);
                                    o[4 * x + 2] = __float_as_uint(__uint_as_float(o[4 * x + 2]) * f.z);
                                    o[4 * x + 3] = __float_as_uint(__uint_as_float(o[4 * x + 3]) * f.w);
                                }
                                const int64_t at = obase + hb * kHD + (dt0 + dd) * 128;
                                if constexpr (kTerms == 1) {
                                    // through shared memory, so that a lane stores 16 bytes of a head (256
                                    // tokens of 1K rows 74.2 -> 72.4 us against a column a lane)
                                    __nv_bfloat16 *const stage =
                                        reinterpret_cast<__nv_bfloat16 *>(sOut + (warp & 3) * kOutBytes);
                                    __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(A.out) + at +
                                                               (lane >> 2) * kHD + (warp & 3) * 32 + (lane & 3) * 8;
#pragma unroll
                                    for (int y = 0; y < 32; y += 16) {
                                        __syncwarp();
#pragma unroll
                                        for (int x = 0; x < 16; ++x)
                                            stage[x * 32 + lane] = __float2bfloat16(__uint_as_float(o[x + y]));
                                        __syncwarp();
#pragma unroll
                                        for (int x = 0; x < 16; x += 8) {
                                            const uint4 v = reinterpret_cast<const uint4 *>(stage)[x * 4 + lane];
                                            if (hb + x + y + (lane >> 2) < hmax) *reinterpret_cast<uint4 *>(dst + (x + y) * kHD) = v;
                                        }
                                    }
                                    __syncwarp();                // (some lanes stored, some did not)
                                } else {
                                    // a column a lane (16 bytes a lane: 83.8 -> 84.6 us for 128-head drafts)
#pragma unroll
                                    for (int x = 0; x < 32; ++x)
                                        if (hb + x < hmax) static_cast<float *>(A.out)[at + x * kHD + dl] = __uint_as_float(o[x]);
                                }
                            }
                        }
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
                while (k.i < nrec && k.c >= S.rec[k.i].c1) {
                    ++k.i;
                    if (k.i < nrec) k.c = S.rec[k.i].c0;
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
                const int n = S.rec[k.i].n, j = k.c * kChunk + 16 * li + rl;
                if (j < n) {
                    const int pg = static_cast<int>(A.page_div.div(j));
                    e.in_page = j - pg * A.L.page_rows;
                    e.page = A.L.table[static_cast<int64_t>(S.rec[k.i].b) * A.L.max_pages + pg];
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
            Cursor cur{0, S.rec[0].c0};
            settle(cur);
            Cursor far = cur;
            const Entry e0 = look_up(far);
            advance(far);
            const Entry e1 = look_up(far);
            advance(far);
            Entry ahead = look_up(far);
            Place now = place(e0), next = place(e1);
            while (cur.i < nrec) {
                const Rec &r = S.rec[cur.i];
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
            if (lane == 0 && lead) raise_status(A.status, bad);
        } else if (warp >= 4) {
            // -------------------------------------------- softmax
            const int q = warp & 3;                  // TMEM lane quarter
            const int hl = q * 16 + (lane & 15);     // head of this lane (two lanes per head)
            const bool upper = lane >= 16;           // rows 32..47 and 24..31 of the chunk, others 0..23
            const bool hv = h0 + hl < H;
            const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
            for (int i = 0; i < nrec; ++i) {
                const int nch = S.rec[i].c1 - S.rec[i].c0;
                if (nch <= 0) {
                    if (S.rec[i].flags & kRecZero) {
                        const int64_t obase = (static_cast<int64_t>(S.rec[i].t) * H + h0) * kHD;
                        for (int x = tid - 128; x < min(kHG, H - h0) * 128 * ndt; x += kSmThreads) {
                            const int64_t at = obase + (x / (128 * ndt)) * kHD + dt0 * 128 + x % (128 * ndt);
                            if (kTerms == 1) static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(0.f);
                            else static_cast<float *>(A.out)[at] = 0.f;
                        }
                    }
                    continue;
                }
                const bool cut = S.rec[i].flags & kRecPart;
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
                            A.part_ml[(static_cast<int64_t>(S.rec[i].slot) * gridDim.y + hg) * kHG + hl] =
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
            S.nrec = 0;
            S.more = 0;
        }
        list_next();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of a cut token:
//   out = sum_s 2^(m_s - M) O_s / (sum_s 2^(m_s - M) l_s [+ 2^(sink - M)]).
// Two shapes: a few tokens cut into up to 152 parts (one long context), and
// many tokens in a few parts each.
struct JoinEntry {
    int t, ns, slot0, split0;
    __device__ int64_t slot(int k) const { return k == 0 ? slot0 : 2 * (split0 + k); }
};

__device__ __forceinline__ JoinEntry join_entry(const PagedArgs &A) {
    const int2 meta = A.meta[blockIdx.x];
    JoinEntry e;
    e.ns = meta.y > kMaxCtas ? 0 : meta.y;
    e.slot0 = meta.x;
    e.split0 = meta.x >> 1;
    // by token: entry x is token x; by CTA: the token stands behind the list
    e.t = blockIdx.x;
    if (A.L.num_tokens > static_cast<int>(gridDim.x)) e.t = A.meta[gridDim.x + blockIdx.x].x;
    return e;
}

// The sink's term 2^(sink - M) of a sum scaled to M >= sink (log2 units): 1 where
// it is the maximum, an infinite one too; NaN stays NaN.
__device__ __forceinline__ float sink_term(float sink, float M) { return sink == M ? 1.f : exp2f(sink - M); }

template <bool kBf16>
__device__ __forceinline__ void join_store(const PagedArgs &A, int64_t at, float x) {
    if (kBf16) static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(x);
    else static_cast<float *>(A.out)[at] = x;
}

// Many parts: a CTA takes four heads of kCols columns; kDeepSub threads share a
// column's parts, eight loads of four heads each in flight (issued before the
// weights are known), and meet in shared memory in order.  One token: 32
// columns, so that every SM reads; a few: a whole 128-column tile.
constexpr int kDeepPer = 8;

template <int kDeepSub, int kCols, bool kBf16>
__global__ void __launch_bounds__(kCols * kDeepSub) join_deep_kernel(const PagedArgs A) {
    __shared__ float wgt[4][kMaxCtas];
    __shared__ float inv_z[4];
    __shared__ float4 red[(kDeepSub - 1) * kCols];
    pdl_wait();
    pdl_launch_dependents();
    const JoinEntry J = join_entry(A);
    const int ns = J.ns;
    if (ns <= 0) return;
    static_assert(kCols * kDeepSub >= 128, "four warps make the weights");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = tid / kCols;
    const int quad = blockIdx.y & 15, tile = blockIdx.y >> 4 & 3, hg = blockIdx.y >> 6;
    const int col = static_cast<int>(blockIdx.z) * kCols + tid % kCols;      // of the tile
    const int groups = static_cast<int>(gridDim.y) >> 6, h0 = hg * kHG + 4 * quad;
    if (h0 >= A.H) return;
    const float4 *const po = A.part_o + tile * (16 * 128) + quad * 128 + col;
    float4 v[kDeepPer];
    auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kDeepPer; ++k)
            if (k0 + k * kDeepSub < ns) v[k] = __ldcg(po + (J.slot(k0 + k * kDeepSub) * groups + hg) * (4 * 16 * 128));
    };
    load(sub);
    if (warp < 4) {                              // the weights of head `warp`
        constexpr int kMl = (kMaxCtas + 31) / 32;
        float2 ml[kMl];
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMl; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            if (lane + 32 * k < ns)
                ml[k] = __ldcg(A.part_ml + (J.slot(lane + 32 * k) * groups + hg) * kHG + 4 * quad + warp);
        }
#pragma unroll
        for (int k = 0; k < kMl; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float sink = A.sinks && h0 + warp < A.H ? A.sinks[h0 + warp] * kLog2e : -INFINITY;
        const float Mall = fmaxf(M, sink);
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < kMl; ++k) {
            const float w = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - Mall);
            if (lane + 32 * k < ns) wgt[warp][lane + 32 * k] = w;
            z += w * ml[k].y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == 0) {
            const bool some = M != -INFINITY;
            if (some) z += sink_term(sink, Mall);
            inv_z[warp] = some ? 1.f / z : 0.f;
        }
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = sub; k0 < ns; k0 += kDeepPer * kDeepSub) {
        if (k0 != sub) load(k0);
#pragma unroll
        for (int k = 0; k < kDeepPer; ++k) {
            const int p = k0 + k * kDeepSub;
            if (p >= ns) break;
            // (heads behind the last hold anything and are not stored)
            acc.x = fmaf(wgt[0][p], v[k].x, acc.x);
            acc.y = fmaf(wgt[1][p], v[k].y, acc.y);
            acc.z = fmaf(wgt[2][p], v[k].z, acc.z);
            acc.w = fmaf(wgt[3][p], v[k].w, acc.w);
        }
    }
    if (sub > 0) red[(sub - 1) * kCols + tid % kCols] = acc;
    __syncthreads();
    if (sub > 0) return;
    for (int j = 0; j + 1 < kDeepSub; ++j) {
        const float4 u = red[j * kCols + tid];
        acc.x += u.x;
        acc.y += u.y;
        acc.z += u.z;
        acc.w += u.w;
    }
    const float o[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (h0 + i < A.H)
            join_store<kBf16>(A, (static_cast<int64_t>(J.t) * A.H + h0 + i) * kHD + tile * 128 + col, o[i] * inv_z[i]);
}

// Few parts: a CTA takes 16 heads of a tile (32 where tokens are many: fewer
// waves of CTAs), a thread two quads of heads of its column at a time, the first
// parts on their way before the weights are made.
constexpr int kWidePer = 3;                      // parts in flight
constexpr int kWideHeads = 32;                   // at most

template <bool kBf16>
__global__ void __launch_bounds__(256) join_wide_kernel(const PagedArgs A) {
    __shared__ float4 wgt[kMaxCtas][kWideHeads / 4];   // scaled by 1 / z
    pdl_wait();
    pdl_launch_dependents();
    const JoinEntry J = join_entry(A);
    const int ns = J.ns;
    if (ns <= 0) return;
    const int tid = threadIdx.x, col = tid & 127, half = tid >> 7;
    const int tile = blockIdx.y & 3, hg = blockIdx.y >> 2, groups = static_cast<int>(gridDim.y) >> 2;
    const int most = kHG / static_cast<int>(gridDim.z);
    const int hb = most * static_cast<int>(blockIdx.z), h0 = hg * kHG + hb;   // first head
    if (h0 >= A.H) return;
    const int heads = min(most, A.H - h0);
    const float4 *const po = A.part_o + tile * (16 * 128) + hb / 4 * 128 + col;
    float4 v[kWidePer][2];
    auto load = [&](int k0, int qd) {                    // quads qd, qd + 1
#pragma unroll
        for (int k = 0; k < kWidePer; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (k0 + k < ns) v[k][e] = __ldcg(po + (J.slot(k0 + k) * groups + hg) * (4 * 16 * 128) + (qd + e) * 128);
    };
    load(0, 2 * half);
    if (tid < most) {
        const float2 *const ml = A.part_ml + hg * kHG + hb + tid;
        const float sink = A.sinks && tid < heads ? A.sinks[h0 + tid] * kLog2e : -INFINITY;
        constexpr int kNear = 6;                 // parts kept in registers
        float2 x[kNear];
#pragma unroll
        for (int k = 0; k < kNear; ++k)
            x[k] = k < ns ? __ldcg(ml + J.slot(k) * groups * kHG) : make_float2(-INFINITY, 0.f);
        float M = x[0].x;
#pragma unroll
        for (int k = 1; k < kNear; ++k) M = fmaxf(M, x[k].x);
        for (int k = kNear; k < ns; ++k) M = fmaxf(M, __ldcg(ml + J.slot(k) * groups * kHG).x);
        const float Mall = fmaxf(M, sink);
        float z = M != -INFINITY ? sink_term(sink, Mall) : 0.f;
        auto put = [&](int k, float2 y) {
            const float w = y.x == -INFINITY ? 0.f : exp2f(y.x - Mall);
            reinterpret_cast<float *>(wgt[k])[tid] = w;
            z += w * y.y;
        };
#pragma unroll
        for (int k = 0; k < kNear; ++k)
            if (k < ns) put(k, x[k]);
        for (int k = kNear; k < ns; ++k) put(k, __ldcg(ml + J.slot(k) * groups * kHG));
        const float f = M != -INFINITY ? 1.f / z : 0.f;
        for (int k = 0; k < ns; ++k) reinterpret_cast<float *>(wgt[k])[tid] *= f;
    }
    __syncthreads();
    const int64_t to = (static_cast<int64_t>(J.t) * A.H + h0) * kHD + tile * 128 + col;
#pragma unroll 1
    for (int qd = 2 * half; 4 * qd < heads; qd += 4) {
        float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        for (int k0 = 0; k0 < ns; k0 += kWidePer) {
            if (k0 > 0 || qd >= 4) load(k0, qd);
#pragma unroll
            for (int k = 0; k < kWidePer; ++k) {
                if (k0 + k >= ns) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float4 w = wgt[k0 + k][qd + e];
                    acc[e].x = fmaf(w.x, v[k][e].x, acc[e].x);
                    acc[e].y = fmaf(w.y, v[k][e].y, acc[e].y);
                    acc[e].z = fmaf(w.z, v[k][e].z, acc[e].z);
                    acc[e].w = fmaf(w.w, v[k][e].w, acc[e].w);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float o[4] = {acc[e].x, acc[e].y, acc[e].z, acc[e].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = 4 * (qd + e) + i;
                if (h < heads) join_store<kBf16>(A, to + static_cast<int64_t>(h) * kHD, o[i]);
            }
        }
    }
}

template <auto kKernel>
cudaError_t launch_one_join(const Launch &lc, const PagedArgs &A, dim3 grid, int threads) {
    const cudaError_t e = prepare_kernel<kKernel>(0);
    return e != cudaSuccess ? e : launch_pdl(kKernel, grid, dim3(threads), 0, lc.stream, A);
}

template <bool kBf16>
cudaError_t launch_join(const Launch &lc, const PagedArgs &A, int entries, int groups, int64_t slots_max) {
    // One token: 8 threads a column where its table has room for few rows (600
    // rows 9.2 us, with 16 threads 10.7), 16 beyond (8,192 rows 14.9 us, with 8
    // threads 15.5).  The length itself is on the device only: in a table of
    // 262,144 rows, 256 rows take 10.0 instead of 9.1 us and 600 rows 10.7.
    if (entries == 1 && slots_max <= 2048)
        return launch_one_join<join_deep_kernel<8, 32, kBf16>>(lc, A, dim3(1, groups * 64, 4), 256);
    if (entries == 1) return launch_one_join<join_deep_kernel<16, 32, kBf16>>(lc, A, dim3(1, groups * 64, 4), 512);
    // Up to 12 tokens, parts by the dozen: a CTA a tile of four heads (8,192 rows
    // each: 2 tokens 18.7 us, with the other kernel 34.5; 8 tokens 29.3 and 34.6; 12
    // tokens 37.5 and 38.8; 16 tokens 44.8 and 42.6; 24 tokens 61.1 and 54.3.  With
    // 128 heads of 2,048 rows the two meet earlier: 4 tokens 18.9 and 23.3, 8
    // tokens 27.1 and 24.1).
    if (entries <= 12) return launch_one_join<join_deep_kernel<4, 128, kBf16>>(lc, A, dim3(entries, groups * 64), 512);
    // beyond, a CTA 16 heads of a tile, or 32 where CTAs are many (24 tokens of
    // 1,500 to 6,000 rows 30.3 us, with 32 heads 32.8; 64 tokens 53.4 and 52.9; 128
    // tokens 91.7, with 16 heads 93.4; 128-head drafts of 64 tokens 76.3 and 77.0)
    const int share = entries * groups >= 96 ? kHG / kWideHeads : 2 * kHG / kWideHeads;
    return launch_one_join<join_wide_kernel<kBf16>>(lc, A, dim3(entries, groups * 4, share), 256);
}

int groups_of(const csa_params_t &p) { return (p.n_heads + kHG - 1) / kHG; }

struct Ws {
    size_t meta, ml, o, total;
};
Ws ws_plan(const csa_params_t &p) {
    const int groups = groups_of(p);
    const size_t slots = 2 * static_cast<size_t>(kMaxCtas / groups) * groups;
    Ws w{};
    w.meta = 0;
    w.ml = (2 * kMaxCtas * sizeof(int2) + 255) / 256 * 256;
    w.o = w.ml + slots * kHG * sizeof(float2);
    w.total = w.o + slots * kHG * kHD * sizeof(float);
    return w;
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
    const int64_t total_rows = (num_pages - 1) * page_stride + L.page_rows;
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
    const Ws w = ws_plan(p);
    uint8_t *wb = static_cast<uint8_t *>(ws);
    PagedArgs A{};
    A.L = L;
    A.H = H;
    A.window = p.window;
    A.ratio = p.ratio;
    A.bf16_out = out_type == CSA_BF16;
    A.scale_log2 = p.scale * kLog2e;
    A.total_rows = static_cast<int32_t>(total_rows);
    A.page_div = FastDiv(L.page_rows);
    A.ratio_div = FastDiv(p.ratio);
    A.swa_div = FastDiv(L.swa_cap > 0 ? L.swa_cap : 1);
    A.num_pages = num_pages;
    A.page_stride = page_stride;
    A.cache = static_cast<const __nv_bfloat16 *>(cache);
    A.sinks = sinks;
    A.out = out;
    A.meta = reinterpret_cast<int2 *>(wb + w.meta);
    A.part_ml = reinterpret_cast<float2 *>(wb + w.ml);
    A.part_o = reinterpret_cast<float4 *>(wb + w.o);
    A.status = status;
    const int ctas = (lc.sm_count < kMaxCtas ? lc.sm_count : kMaxCtas) / groups;
    for (int i = 0; i < 3; ++i) A.split_div[i] = FastDiv(ctas >> i);
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
