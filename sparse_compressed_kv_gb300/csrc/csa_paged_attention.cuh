// csa_paged_attention.cuh -- what the attention kernels over paged caches share
// (bf16 rows: csa_paged_attention.cu, e4m3 rows: csa_paged_attention_fp8.cu):
// the arguments, what a token attends, the division of all tokens' chunks over
// the CTAs, the workspace, and the kernels that join the parts of a cut token.
#pragma once

#include "csa_device.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kHG = 64;                         // heads per CTA
constexpr int kEpThreads = 128;                 // four warps: the epilogue, which also issue the products
constexpr int kBarSm = 1;
// of an epilogue warp, on their way to a bf16 output: 32 columns of some heads
constexpr int staged_bytes(int heads) { return heads * 32 * 2; }
constexpr int kMaxCtas = 152;                   // CTAs of the grid at most (sizes the workspace)

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

// Chunks after which a segment of nch chunks rounds its accumulator into the
// partial: equal stretches of at most kMost.
template <int kMost>
__device__ __forceinline__ int flush_every(int nch) {
    const int n = (nch + kMost - 1) / kMost;
    return n > 1 ? (nch + n - 1) / n : nch;
}

// The division of the work, the part in shared memory: counts, and the list of
// the CTA's next segments.
template <int kMaxRec>
struct WorkSmem {
    int32_t nrec, more;
    int32_t t0, s0;
    int2 wsum[16];               // of a warp: cost, most chunks of a token
    Rec rec[kMaxRec];
};

// Every CTA (of kThreads threads) counts the chunks of kChunk row slots of all tokens for itself and
// takes an equal contiguous range of them, kMaxRec segments at a time; a segment costs kSegCost chunks more.
// Used by all threads: count(), a barrier, divide(), first_list(), then next_list()
// between barriers while S.more is set.  (The layout is read before the wait for
// the preceding kernel, as everywhere in this library.)
template <int kThreads, int kMaxRec, int kChunk, int kSegCost, int kCutAbove>
struct Work {
    const PagedArgs &A;
    WorkSmem<kMaxRec> &S;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = gridDim.x, T = A.L.num_tokens;
    const bool by_token = T <= G;
    const int tps = max(1, T / A.L.num_seqs);
    const int per = (T + kThreads - 1) / kThreads;
    const int ta = min(T, tid * per), te = min(T, ta + per);
    Rec own{};
    int own_c = 0, own_bad = 0;
    int cost = 0, incl = 0, base = 0;
    bool direct = false, snap = false, lead = false;
    int split = 0, share = 0, ua = 0, ub = 0, t0 = 0, s0 = 0;
    int ndt = 4, dt0 = 0;                // 128-column tiles of this CTA, the first

    __device__ __forceinline__ Work(const PagedArgs &args, WorkSmem<kMaxRec> &smem) : A(args), S(smem) {}

    // (a token's slots may end 57 below 2^31: rounded up they pass 31 bits)
    static __device__ __forceinline__ int chunks(const Rec &r) {
        return r.b < 0 ? 0 : static_cast<int>((static_cast<uint32_t>(rec_slots(r)) + kChunk - 1u) / kChunk);
    }
    static __device__ __forceinline__ int cost_of(int c) { return c > 0 ? c + kSegCost : 1; }

    // Chunks and costs of all tokens, a contiguous run of tokens per thread; with
    // one token a thread its record stays in registers.
    __device__ __forceinline__ void count() {
        int maxc = 0;
        for (int t = ta; t < te; ++t) {
            own = token_rec(A, t, tps, own_bad);
            own_c = chunks(own);
            cost += cost_of(own_c);
            maxc = max(maxc, own_c);
        }
        incl = cost;
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
    }

    // This CTA's range, and the token it begins with.
    __device__ __forceinline__ void divide() {
        int U = 0, maxc = 0;                 // units of all tokens
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w == warp) base = U;         // units in front of this warp
            U += S.wsum[w].x;
            maxc = max(maxc, S.wsum[w].y);
        }
        // Tokens are cut only where that shortens the longest CTA by more than
        // the partials and their join cost: otherwise CTA c takes token c (T <= G),
        // or the tokens that begin in its range.
        direct = T <= G && maxc <= static_cast<int>(A.split_div[0].div(U)) + kCutAbove;
        snap = direct || (T > G && maxc <= kCutAbove);
        // few CTAs at work: 2 or 4 of them share a range, each with all of its
        // logits and weights and its share of the 512 columns: the last products
        // and the partial (32 bytes a cycle and SM) are that much shorter (bf16 rows,
        // 8,192 of them, three chunks for two CTAs 14.8 us, two for one 15.3)
        int dlog = 0;
        if (direct) dlog = T * 4 <= G ? 2 : T * 2 <= G ? 1 : 0;
        else if (!snap && T <= G) dlog = U <= G / 4 ? 2 : U <= G + G / 3 ? 1 : 0;
        const int dparts = 1 << dlog;
        split = static_cast<int>(blockIdx.x) >> dlog;
        ndt = 4 >> dlog;
        dt0 = (static_cast<int>(blockIdx.x) & (dparts - 1)) * ndt;
        // equal ranges of `share` units, the last ones shorter or empty: as few parts
        // as the longest range allows
        share = static_cast<int>(A.split_div[dlog].div(U + (G >> dlog) - 1));
        ub = split < T ? 1 : 0;
        if (!direct) {
            ua = min(split * share, U);
            ub = min(ua + share, U);
        }
        lead = blockIdx.y == 0 && dt0 == 0;      // reports errors, writes the join's list
        // The first token of the range: the one that holds unit ua, or (whole
        // tokens only) the first that begins at or behind it.
        if (direct) {
            if (tid == 0) S.t0 = split;
        } else {
            int s = base + incl - cost;
            for (int t = ta; t < te; ++t) {
                int bad;
                const int c = per == 1 ? own_c : chunks(token_rec(A, t, tps, bad));
                const int e = s + cost_of(c);
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
                s += cost_of(chunks(token_rec(A, t, tps, bad)));
            }
            __syncthreads();
        }
        t0 = S.t0;
        s0 = S.s0;
    }

    // Lists the segment of one token (whose units begin at s) as entry `at`.
    // Returns the token's entry for the join; `owner`: its first chunk is here.
    __device__ __forceinline__ int2 list(Rec &r, int c, int s, int at, bool &owner) {
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
            S.s0 = s + cost_of(c);
        }
        return m;
    }

    __device__ __forceinline__ void report(const Rec &r, int bad, int2 m) {
        raise_status(A.status, bad);
        if (by_token) {
            A.meta[r.t] = m;
        } else if (m.y > 0) {
            A.meta[split] = m;
            A.meta[G + split] = make_int2(r.t, 0);
        }
    }

    // The next segments: thread i lists token t0 + i.
    __device__ __forceinline__ void next_list() {
        Rec r{};
        int bad = 0, c = 0, w = 0;
        const bool in = tid < kMaxRec && t0 + tid < T && ub > ua;
        if (in) {
            r = token_rec(A, t0 + tid, tps, bad);
            c = chunks(r);
            w = cost_of(c);
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
    }

    // The first segments, from the registers where they can be, around the wait for
    // the preceding kernel.
    __device__ __forceinline__ void first_list() {
        if (per == 1) {
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
            next_list();
        }
    }

    // Behind a list that was worked off: on to the next tokens.
    __device__ __forceinline__ void advance() {
        t0 += kMaxRec;
        s0 = S.s0;
    }
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

// Unswizzled K-major operand: atoms of 8 rows x 16 bytes, 128 contiguous bytes
// each, `lbo` apart along K and `sbo` along the rows.
__device__ __forceinline__ uint64_t atom_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return sw128_desc(saddr, lbo, sbo) & ~(static_cast<uint64_t>(7u) << 61);
}

// a byte offset as a step of a descriptor's start-address field (every shared
// address is below 256 KiB, so the field never carries)
__device__ __forceinline__ constexpr uint64_t off(uint32_t bytes) { return bytes >> 4; }

// O^T of a stretch into the partial, or the output, by the epilogue's warps: tile by
// tile, each handed back to the products (by `ofree`, if any) once it is in registers.
// A warp has the columns of its quarter and the heads hb0 .. hb1 - 1 (multiples of 32)
// below hmax.
//   o_tmem  the first tile's first column, in this warp's lanes; each tile has 64
//           columns (heads), the first kWide ones 64 more that are added to them
//   add     the partial holds earlier stretches, to be scaled by `flush`
//   sOut    staged_bytes(kStagedHeads) of this warp's own, for a bf16 output
//   part    leave (O, m, l); otherwise the output, scaled by `fin`
template <bool kBf16, int kWide, int kStagedHeads>
__device__ __forceinline__ void drain_stretch(const PagedArgs &A, uint32_t o_tmem, const float *fin,
                                              const float *flush, uint64_t *ofree, uint8_t *sOut, int dt0,
                                              int ndt, int hb0, int hb1, int hmax, int64_t obase, int64_t pslot, bool add,
                                              bool part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dl = (warp & 3) * 32 + lane;       // column of a tile
#pragma unroll 1
    for (int dd = 0; dd < ndt; ++dd) {
        // one column per lane; a partial keeps four heads together,
        // so that a warp stores 512 contiguous bytes
        float4 *const pd = A.part_o + (pslot * 4 + dt0 + dd) * (16 * 128) + dl;
#pragma unroll 1
        for (int hb = hb0; hb < hb1; hb += 32) {
            if (hb >= hmax) {                    // (hb0: nothing to do)
                if (ofree && hb == hb0) mbar_arrive(&ofree[dd]);
                break;
            }
            uint32_t o[32];
            const uint32_t oc = o_tmem + kHG * (dd + (dd < kWide ? dd : kWide)) + hb;
            tmem_ld16_raw(oc, *reinterpret_cast<uint32_t(*)[16]>(o));
            tmem_ld16_raw(oc + 16, *reinterpret_cast<uint32_t(*)[16]>(o + 16));
            float4 *const pq = pd + hb / 4 * 128;
            if (dd < kWide) {
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
                    const float4 f = *reinterpret_cast<const float4 *>(flush + hb + 4 * x);
                    o[4 * x] = __float_as_uint(fmaf(old[x].x, f.x, __uint_as_float(o[4 * x])));
                    o[4 * x + 1] = __float_as_uint(fmaf(old[x].y, f.y, __uint_as_float(o[4 * x + 1])));
                    o[4 * x + 2] = __float_as_uint(fmaf(old[x].z, f.z, __uint_as_float(o[4 * x + 2])));
                    o[4 * x + 3] = __float_as_uint(fmaf(old[x].w, f.w, __uint_as_float(o[4 * x + 3])));
                }
            }
            tmem_wait_ld();
            if (hb + 32 >= min(hb1, hmax)) { // the tile is in registers
                tc_fence_before();
                if (ofree) mbar_arrive(&ofree[dd]);
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
                const float4 f = *reinterpret_cast<const float4 *>(fin + hb + 4 * x);
                o[4 * x] = __float_as_uint(__uint_as_float(o[4 * x]) * f.x);
                o[4 * x + 1] = __float_as_uint(__uint_as_float(o[4 * x + 1]) * f.y);
                o[4 * x + 2] = __float_as_uint(__uint_as_float(o[4 * x + 2]) * f.z);
                o[4 * x + 3] = __float_as_uint(__uint_as_float(o[4 * x + 3]) * f.w);
            }
            const int64_t at = obase + hb * kHD + (dt0 + dd) * 128;
            if constexpr (kBf16) {
                // through shared memory, so that a lane stores 16 bytes of a head (256
                // tokens of 1K rows 74.2 -> 72.4 us against a column a lane)
                __nv_bfloat16 *const stage =
                    reinterpret_cast<__nv_bfloat16 *>(sOut);
                __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(A.out) + at +
                                           (lane >> 2) * kHD + (warp & 3) * 32 + (lane & 3) * 8;
#pragma unroll
                for (int y = 0; y < 32; y += kStagedHeads) {
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < kStagedHeads; ++x)
                        stage[x * 32 + lane] = __float2bfloat16(__uint_as_float(o[x + y]));
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < kStagedHeads; x += 8) {
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

// rows from the pool's first to the last of its last page
inline int64_t paged_rows(const csa_paged_layout_t &L, int64_t num_pages, int64_t page_stride) {
    return (num_pages - 1) * page_stride + L.page_rows;
}

// The arguments but for the rows themselves; split_div[0].d is the number of CTAs
// a group of heads has.
PagedArgs paged_args(const Launch &lc, const csa_paged_layout_t &L, const csa_params_t &p, int64_t num_pages,
                     int64_t page_stride, const float *sinks, csa_type_t out_type, void *out,
                     int32_t *status, void *ws) {
    const Ws w = ws_plan(p);
    uint8_t *wb = static_cast<uint8_t *>(ws);
    PagedArgs A{};
    A.L = L;
    A.H = p.n_heads;
    A.window = p.window;
    A.ratio = p.ratio;
    A.bf16_out = out_type == CSA_BF16;
    A.scale_log2 = p.scale * kLog2e;
    A.total_rows = static_cast<int32_t>(paged_rows(L, num_pages, page_stride));
    A.page_div = FastDiv(L.page_rows);
    A.ratio_div = FastDiv(p.ratio);
    A.swa_div = FastDiv(L.swa_cap > 0 ? L.swa_cap : 1);
    A.num_pages = num_pages;
    A.page_stride = page_stride;
    A.sinks = sinks;
    A.out = out;
    A.meta = reinterpret_cast<int2 *>(wb + w.meta);
    A.part_ml = reinterpret_cast<float2 *>(wb + w.ml);
    A.part_o = reinterpret_cast<float4 *>(wb + w.o);
    A.status = status;
    const int ctas = (lc.sm_count < kMaxCtas ? lc.sm_count : kMaxCtas) / groups_of(p);
    for (int i = 0; i < 3; ++i) A.split_div[i] = FastDiv(ctas >> i);
    return A;
}

}  // namespace
}  // namespace csa
