// csa_paged.cu -- paged caches: the C entry points, the page plan and the
// append (include/csa.h, "Paged caches").  The attention over the pages is in
// csa_paged_attention.cu.
#include <math.h>

#include "csa_device.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

// ---------------------------------------------------------------- page plan

// Four exclusive prefix sums over the requests (tokens, new blocks, pages
// taken, pages given back) fix everything.  Every CTA makes the sums for itself
// from the 12 bytes per request (no exchange between CTAs), keeps them in
// shared memory and writes its share of the outputs.  The kernel is a chain of
// latencies and of instructions, not of bytes: small CTAs, each thread summing
// several requests, divisions by products, 32-bit sums.  In a decode step,
// where every request brings a few tokens, the thread that has a request writes
// all of its entries; with prompts among them each output entry is computed by
// itself, its request found by bisection.  Replayed from a graph 32 requests take
// 3.9 us, 1,024 requests 5.9, 256 requests with 77K tokens of prompts 6.9 (an
// empty launch about 2); called in a stream 4.3, 5.8 and 6.8.
constexpr int kPlanThreads = 256;
constexpr int kPlanBatch = 4;     // requests a thread loads at a time
constexpr int kPlanMaxSeqs = 8192;
constexpr int64_t kPlanMaxLen = int64_t(1) << 48;
constexpr uint32_t kPlanFew = 8;  // tokens a request, at most, for a thread to write them in turn

struct PlanArgs {
    csa_page_plan_t P;
    FastDiv ratio, page_rows, swa_cap, num_pages;
};

struct Req {
    int64_t len, end, old_rows;
    uint32_t add, new_rows;       // tokens and blocks that the step brings
    int32_t old_pages, pages;     // (saturated: more than the table has is refused)
    bool over;
};

__device__ __forceinline__ int32_t plan_pages(const PlanArgs &A, int64_t rows) {
    const int64_t n = A.page_rows.div64(rows + A.P.page_rows - 1);
    return n > INT32_MAX ? INT32_MAX : static_cast<int32_t>(n);
}

__device__ __forceinline__ Req plan_request(const PlanArgs &A, int64_t len, int32_t nl) {
    Req r;
    r.len = len;
    r.over = nl < 0;
    r.add = nl > 0 ? nl : 0;
    r.end = r.over ? 0 : len + r.add;
    r.old_rows = A.ratio.div64(len);
    // len = old_rows ratio + rest; the sum below fits 32 bits
    r.new_rows = A.ratio.div(static_cast<uint32_t>(len - r.old_rows * A.P.ratio) + r.add);
    r.old_pages = plan_pages(A, r.old_rows);
    r.pages = plan_pages(A, r.old_rows + r.new_rows);
    return r;
}

struct Sums {
    uint32_t tok, row, need, rel;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return {a.tok + b.tok, a.row + b.row, a.need + b.need, a.rel + b.rel};
}
__device__ __forceinline__ Sums operator-(const Sums &a, const Sums &b) {
    return {a.tok - b.tok, a.row - b.row, a.need - b.need, a.rel - b.rel};
}

__device__ __forceinline__ Sums plan_sums(const Req &r) {
    if (r.over) return {0, 0, 0, static_cast<uint32_t>(r.old_pages)};
    return {r.add, r.new_rows, static_cast<uint32_t>(r.pages - r.old_pages), 0};
}

__device__ __forceinline__ Sums scan_warp(Sums v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums u{__shfl_up_sync(0xffffffffu, v.tok, o), __shfl_up_sync(0xffffffffu, v.row, o),
                     __shfl_up_sync(0xffffffffu, v.need, o), __shfl_up_sync(0xffffffffu, v.rel, o)};
        if (lane >= o) v = v + u;
    }
    return v;
}

// The last request whose range starts at or before i (ranges of requests
// without elements are empty, so the last one that starts there holds i).
template <uint32_t Sums::*kField>
__device__ __forceinline__ int plan_find(const Sums *off, int n, uint32_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid].*kField <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs A, int32_t *status) {
    extern __shared__ Sums off[];                // [B] exclusive
    const csa_page_plan_t &P = A.P;
    const int B = P.num_seqs;
    constexpr int kWarps = kPlanThreads / 32;
    __shared__ Sums warp_sum[kWarps];
    __shared__ uint32_t warp_tok[kWarps], warp_rel[kWarps], warp_bad[kWarps], warp_most[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();      // (and no early start for what follows: it may read the maps before its own wait)
    const int64_t head = P.free_pos[0], tail = P.free_pos[1], N = P.num_pages;

    // this thread's contiguous run of requests
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    Sums mine{0, 0, 0, 0};
    // Sums are 32-bit; whether one passes 2^31 (more than any capacity) shows in
    // the sums of the upper halves of what is added: where those stay
    // below 2^15, 8192 requests add less than 2^32.
    uint32_t bad = 0, most = 0, tok_hi = 0, rel_hi = 0;
    for (int b = b0; b < b1; b += kPlanBatch) {
        int64_t len[kPlanBatch];
        int32_t nl[kPlanBatch];
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            len[k] = b + k < b1 ? P.seq_len[b + k] : 0;
            nl[k] = b + k < b1 ? P.new_len[b + k] : 0;
        }
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            if (b + k >= b1) break;
            off[b + k] = mine;
            if (len[k] < 0 || len[k] >= kPlanMaxLen || nl[k] < -1) {
                bad |= CSA_DEV_BAD_LENGTH;
                continue;
            }
            const Req r = plan_request(A, len[k], nl[k]);
            if (r.old_pages > P.max_pages || r.pages > P.max_pages) bad |= CSA_DEV_CAPACITY;
            const Sums v = plan_sums(r);
            mine = mine + v;
            most = max(most, r.add);
            tok_hi += v.tok >> 16;
            rel_hi += v.rel >> 16;
        }
    }
    const Sums incl = scan_warp(mine, lane);
    bad = __reduce_or_sync(0xffffffffu, bad);
    most = __reduce_max_sync(0xffffffffu, most);
    tok_hi = __reduce_add_sync(0xffffffffu, tok_hi);
    rel_hi = __reduce_add_sync(0xffffffffu, rel_hi);
    if (lane == 31) {
        warp_sum[warp] = incl;
        warp_bad[warp] = bad;
        warp_most[warp] = most;
        warp_tok[warp] = tok_hi;
        warp_rel[warp] = rel_hi;
    }
    __syncthreads();
    Sums base{0, 0, 0, 0}, total{0, 0, 0, 0};
    bad = most = tok_hi = rel_hi = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) base = total;
        total = total + warp_sum[w];
        bad |= warp_bad[w];
        most = max(most, warp_most[w]);
        tok_hi += warp_tok[w];
        rel_hi += warp_rel[w];
    }
    const bool wide = tok_hi >= 1u << 15;        // (blocks and pages are no more than tokens)
    if (head < 0 || tail < head || tail - head > N || tail >= kPlanMaxLen) bad |= CSA_DEV_BAD_LAYOUT;
    else if (wide || total.need > tail - head) bad |= CSA_DEV_CAPACITY;
    else if (rel_hi >= 1u << 15 || tail + total.rel - head > N) bad |= CSA_DEV_BAD_LAYOUT;   // more pages than the pool has
    if (wide || total.tok > P.tok_cap || total.row > P.row_cap) bad |= CSA_DEV_CAPACITY;
    const bool ok = bad == 0;
    if (blockIdx.x == 0 && tid == 0) raise_status(status, static_cast<int>(bad));
    if (!ok) total = Sums{0, 0, 0, 0};           // no tokens, blocks or pages
    const Sums front = base + incl - mine;
    for (int b = b0; b < b1; ++b) off[b] = ok ? off[b] + front : Sums{0, 0, 0, 0};
    __syncthreads();

    // place k of the ring, k < N: at most once around
    const int64_t h0 = ok ? A.num_pages.mod64(head) : 0, t0 = ok ? A.num_pages.mod64(tail) : 0;
    auto ring = [&](int64_t from, uint32_t k) {
        const int64_t i = from + k;
        return P.free_ring + (i >= N ? i - N : i);
    };
    auto put_token = [&](uint32_t i, int b, int64_t pos, int64_t end) {
        P.tok_seq[i] = b;
        P.tok_pos[i] = pos;
        P.swa_slot[i] = pos >= end - P.swa_cap ? static_cast<int64_t>(b) * P.swa_cap + A.swa_cap.mod64(pos) : -1;
    };
    // a page number that the table or the ring should not hold
    int wrong = 0;
    auto known = [&](int32_t page) {
        const bool ok = page >= 0 && page < N;
        if (!ok) wrong = CSA_DEV_BAD_INDEX;
        return ok;
    };
    // new block k of request b, whose new pages start at place `need`
    auto put_row = [&](uint32_t i, int b, const Req &r, uint32_t k, uint32_t need) {
        const int64_t g = r.old_rows + k;
        const int32_t pg = static_cast<int32_t>(A.page_rows.div64(g));
        if (!CSA_CHECK(pg >= 0 && pg < P.max_pages && pg < r.pages, status)) return;
        const int32_t page = pg < r.old_pages ? P.table[static_cast<int64_t>(b) * P.max_pages + pg]
                                              : *ring(h0, need + (pg - r.old_pages));
        P.row_slot[i] = known(page) ? static_cast<int64_t>(page) * P.page_rows + (g - static_cast<int64_t>(pg) * P.page_rows)
                                    : -1;
    };
    const bool few = most <= kPlanFew;
    const uint32_t step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
    for (uint32_t b = first; b < static_cast<uint32_t>(B); b += step) {
        const Sums at = off[b];
        P.tok_off[b] = at.tok;
        P.row_off[b] = at.row;
        const int64_t len = P.seq_len[b];
        Req r{};
        if (ok) r = plan_request(A, len, P.new_len[b]);
        const int64_t end = ok ? r.end : len;
        P.seq_len_out[b] = end;
        P.row_len[b] = ok ? (r.over ? 0 : r.old_rows + r.new_rows) : end > 0 ? end / P.ratio : 0;
        P.swa_first_pos[b] = end > P.swa_cap ? end - P.swa_cap : 0;
        if (!ok || !few || r.over) continue;
        for (uint32_t k = 0; k < r.add; ++k) put_token(at.tok + k, b, len + k, end);
        for (uint32_t k = 0; k < r.new_rows; ++k) put_row(at.row + k, b, r, k, at.need);
        for (int32_t pg = r.old_pages; pg < r.pages; ++pg)
            P.table[static_cast<int64_t>(b) * P.max_pages + pg] = *ring(h0, at.need + (pg - r.old_pages));
    }
    if (first == 0) {
        P.tok_off[B] = total.tok;
        P.row_off[B] = total.row;
        P.free_pos_out[0] = head + total.need;
        P.free_pos_out[1] = tail + total.rel;
    }
    if (!few) {
        for (uint32_t i = first; i < total.tok; i += step) {
            const int b = plan_find<&Sums::tok>(off, B, i);
            const int64_t len = P.seq_len[b];
            put_token(i, b, len + (i - off[b].tok), len + P.new_len[b]);
        }
        for (uint32_t i = first; i < total.row; i += step) {
            const int b = plan_find<&Sums::row>(off, B, i);
            put_row(i, b, plan_request(A, P.seq_len[b], P.new_len[b]), i - off[b].row, off[b].need);
        }
        for (uint32_t i = first; i < total.need; i += step) {
            const int b = plan_find<&Sums::need>(off, B, i);
            const int32_t pg = plan_pages(A, A.ratio.div64(P.seq_len[b])) + static_cast<int32_t>(i - off[b].need);
            if (CSA_CHECK(pg < P.max_pages, status))
                P.table[static_cast<int64_t>(b) * P.max_pages + pg] = *ring(h0, i);
        }
    }
    for (uint32_t i0 = first; i0 < total.rel; i0 += kPlanBatch * step) {
        int32_t page[kPlanBatch];
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            const uint32_t i = i0 + k * step;
            if (i >= total.rel) break;
            const int b = plan_find<&Sums::rel>(off, B, i);
            page[k] = P.table[static_cast<int64_t>(b) * P.max_pages + (i - off[b].rel)];
        }
#pragma unroll
        for (int k = 0; k < kPlanBatch; ++k) {
            if (i0 + k * step >= total.rel) break;
            (void)known(page[k]);
            *ring(t0, i0 + k * step) = page[k];
        }
    }
    for (int64_t i = static_cast<int64_t>(total.tok) + first; i < P.tok_cap; i += step) {
        P.tok_seq[i] = -1;
        P.tok_pos[i] = -1;
        P.swa_slot[i] = -1;
    }
    for (int64_t i = static_cast<int64_t>(total.row) + first; i < P.row_cap; i += step) P.row_slot[i] = -1;
    raise_status(status, wrong);
    __threadfence();
}

// ---------------------------------------------------------------- append

struct AppendJob {
    const char *rows;
    const int64_t *slots;
    char *cache;
    int64_t row_pitch, page_stride;
    FastDiv pieces, page_rows;                         // 16-byte pieces a row
    uint32_t slot_end, row_bytes;                      // slot_end: num_pages * page_rows
};
struct AppendArgs {
    AppendJob job[CSA_MAX_APPEND_JOBS];
    int64_t start[CSA_MAX_APPEND_JOBS + 1];            // first piece of each pair, all of them
    int32_t num_jobs;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendPer = 4;     // pieces a thread has in flight

// A plain copy: bound by DRAM when large (354 MB in 57.9 us: 90% of the copy
// rate), by two round trips when small (2.2 us replayed from a graph, 4.1 called
// in a stream).  The 16-byte pieces of all pairs are one index range; a
// thread loads four pieces and their slots before it stores the first.
// Index arithmetic is 32-bit inside a pair: in 64 bits its divisions, four a
// piece, took longer than the copy (79.8 us).
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs A, int32_t *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t all = A.start[A.num_jobs];
    const int64_t step = static_cast<int64_t>(gridDim.x) * kAppendThreads * kAppendPer;
    int bad = 0;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kAppendThreads * kAppendPer + threadIdx.x; i0 < all;
         i0 += step) {
        uint4 v[kAppendPer];
        int64_t slot[kAppendPer];
        uint32_t c[kAppendPer];
        int j[kAppendPer];
#pragma unroll
        for (int k = 0; k < kAppendPer; ++k) {
            const int64_t i = i0 + k * kAppendThreads;
            slot[k] = -1;
            if (i >= all) continue;
            j[k] = 0;
#pragma unroll
            for (int q = 1; q < CSA_MAX_APPEND_JOBS; ++q)
                if (q < A.num_jobs && i >= A.start[q]) j[k] = q;
            const AppendJob &J = A.job[j[k]];
            const uint32_t e = static_cast<uint32_t>(i - A.start[j[k]]);
            const uint32_t row = J.pieces.div(e);
            c[k] = (e - row * J.pieces.d) * 16;
            slot[k] = J.slots[row];
            v[k] = __ldcs(reinterpret_cast<const uint4 *>(J.rows + row * J.row_pitch + c[k]));
        }
#pragma unroll
        for (int k = 0; k < kAppendPer; ++k) {
            if (slot[k] < 0) continue;
            const AppendJob &J = A.job[j[k]];
            if (slot[k] >= J.slot_end) {
                bad = CSA_DEV_BAD_INDEX;
                continue;
            }
            const uint32_t s = static_cast<uint32_t>(slot[k]), page = J.page_rows.div(s);
            const int64_t at = page * J.page_stride + (s - page * J.page_rows.d);
            *reinterpret_cast<uint4 *>(J.cache + at * J.row_bytes + c[k]) = v[k];
        }
    }
    raise_status(status, bad);
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t k2G = int64_t(1) << 31;

struct Range {
    const void *p;
    int64_t bytes;
};

// Whether one of the first `written` arrays shares memory with any other array.
template <int kN>
bool overlapping(const Range (&r)[kN], int written) {
    for (int i = 0; i < written; ++i) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p);
        if (!r[i].p || r[i].bytes <= 0) continue;
        for (int j = i + 1; j < kN; ++j) {
            const uintptr_t b = reinterpret_cast<uintptr_t>(r[j].p);
            if (!r[j].p || r[j].bytes <= 0) continue;
            if (a < b + r[j].bytes && b < a + r[i].bytes) return true;
        }
    }
    return false;
}

csa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

csa_status_t check_paged(const csa_paged_layout_t *L, const csa_params_t *p) {
    if (!L || !p) return CSA_ERR_INVALID_ARGUMENT;
    if (p->hd != kHD) return CSA_ERR_UNSUPPORTED;
    if (p->n_heads < 1 || p->window < 0 || p->ratio < 1 || !isfinite(p->scale))
        return CSA_ERR_INVALID_ARGUMENT;
    if (p->n_heads > 128) return CSA_ERR_UNSUPPORTED;
    if (L->num_seqs < 1 || L->num_tokens < 0 || L->page_rows < 1 || L->max_pages < 1)
        return CSA_ERR_INVALID_ARGUMENT;
    if (L->num_tokens > kPagedMaxTokens) return CSA_ERR_UNSUPPORTED;
    const int64_t rows = static_cast<int64_t>(L->max_pages) * L->page_rows + p->window;
    if (rows >= k2G - 64 || rows * L->num_tokens >= int64_t(1) << 36) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_page_plan(const csa_page_plan_t *plan, int32_t *dev_status,
                                      void *stream) {
    if (!plan) return CSA_ERR_INVALID_ARGUMENT;
    const csa_page_plan_t &P = *plan;
    if (P.num_seqs < 1 || P.ratio < 1 || P.page_rows < 1 || P.max_pages < 1 || P.num_pages < 1 ||
        P.swa_cap < 1 || P.tok_cap < 0 || P.row_cap < 0)
        return CSA_ERR_INVALID_ARGUMENT;
    if (P.num_seqs > kPlanMaxSeqs || P.num_pages >= k2G || P.num_pages * P.page_rows >= k2G ||
        P.tok_cap >= k2G || P.row_cap >= k2G)
        return CSA_ERR_UNSUPPORTED;
    const void *const need[] = {P.seq_len, P.new_len, P.table, P.free_ring, P.free_pos,
                                P.seq_len_out, P.row_len, P.swa_first_pos, P.free_pos_out,
                                P.tok_off, P.row_off, dev_status};
    for (const void *p : need)
        if (!p) return CSA_ERR_INVALID_ARGUMENT;
    if (P.tok_cap > 0 && (!P.tok_seq || !P.tok_pos || !P.swa_slot)) return CSA_ERR_INVALID_ARGUMENT;
    if (P.row_cap > 0 && !P.row_slot) return CSA_ERR_INVALID_ARGUMENT;
    const void *const wide[] = {P.seq_len, P.free_pos, P.seq_len_out, P.row_len, P.swa_first_pos,
                                P.free_pos_out, P.tok_off, P.row_off, P.tok_pos, P.swa_slot,
                                P.row_slot};
    for (const void *p : wide)
        if (p && !aligned(p, 8)) return CSA_ERR_INVALID_ARGUMENT;
    const void *const narrow[] = {P.new_len, P.table, P.free_ring, P.tok_seq, dev_status};
    for (const void *p : narrow)
        if (p && !aligned(p, 4)) return CSA_ERR_INVALID_ARGUMENT;
    // every CTA reads the inputs, some of them again for each output, while
    // others write: what is written shares memory with nothing else
    const int64_t B = P.num_seqs;
    const Range arrays[] = {{P.table, B * P.max_pages * 4}, {P.free_ring, P.num_pages * 4},
                            {P.seq_len_out, B * 8}, {P.row_len, B * 8}, {P.swa_first_pos, B * 8},
                            {P.free_pos_out, 16}, {P.tok_off, (B + 1) * 8}, {P.row_off, (B + 1) * 8},
                            {P.tok_seq, P.tok_cap * 4}, {P.tok_pos, P.tok_cap * 8},
                            {P.swa_slot, P.tok_cap * 8}, {P.row_slot, P.row_cap * 8}, {dev_status, 4},
                            {P.seq_len, B * 8}, {P.new_len, B * 4}, {P.free_pos, 16}};
    if (overlapping(arrays, 13)) return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    if (prepare_kernel<page_plan_kernel>(kPlanMaxSeqs * sizeof(Sums)) != cudaSuccess) return CSA_ERR_CUDA;
    const size_t smem = static_cast<size_t>(P.num_seqs) * sizeof(Sums);
    // a request or two output entries a thread, one CTA an SM at most; and some
    // for the pages that requests may give back (how many is on the device)
    int64_t items = P.tok_cap > P.row_cap ? P.tok_cap : P.row_cap;
    items = (items + 1) / 2 > P.num_seqs ? (items + 1) / 2 : P.num_seqs;
    int64_t grid = (items + kPlanThreads - 1) / kPlanThreads;
    const int64_t held = static_cast<int64_t>(P.num_seqs) * P.max_pages;
    const int64_t back = (held < P.num_pages ? held : P.num_pages) / (16 * kPlanThreads);
    if (grid < back) grid = back;
    if (grid > sms) grid = sms;
    const PlanArgs A{P, FastDiv(P.ratio), FastDiv(P.page_rows), FastDiv(P.swa_cap),
                     FastDiv(static_cast<uint32_t>(P.num_pages))};
    return cuda_status(launch_pdl(page_plan_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPlanThreads), smem,
                                  static_cast<cudaStream_t>(stream), A, dev_status));
}

extern "C" csa_status_t csa_paged_append(const csa_append_job_t *jobs, int32_t num_jobs,
                                         int32_t *dev_status, void *stream) {
    if (!jobs || num_jobs < 1 || !dev_status) return CSA_ERR_INVALID_ARGUMENT;
    if (num_jobs > CSA_MAX_APPEND_JOBS) return CSA_ERR_UNSUPPORTED;
    AppendArgs A{};
    for (int j = 0; j < num_jobs; ++j) {
        const csa_append_job_t &J = jobs[j];
        if (J.num_rows < 0 || J.row_bytes < 16 || J.row_bytes % 16 || J.page_rows < 1 ||
            J.num_pages < 1 || J.page_stride < J.page_rows || J.row_pitch < J.row_bytes ||
            J.row_pitch % 16)
            return CSA_ERR_INVALID_ARGUMENT;
        if (J.num_pages >= k2G || J.num_pages * J.page_rows >= k2G || J.row_bytes > 65536 ||
            J.page_stride >= k2G || J.num_rows >= k2G || J.num_rows * J.row_bytes >= int64_t(1) << 36)
            return CSA_ERR_UNSUPPORTED;
        if (J.num_rows == 0) continue;
        if (!J.rows || !J.slots || !J.cache) return CSA_ERR_INVALID_ARGUMENT;
        if (!aligned(J.rows, 16) || !aligned(J.cache, 16) || !aligned(J.slots, 8))
            return CSA_ERR_INVALID_ARGUMENT;
        AppendJob &K = A.job[A.num_jobs];
        K.rows = static_cast<const char *>(J.rows);
        K.slots = J.slots;
        K.cache = static_cast<char *>(J.cache);
        K.row_pitch = J.row_pitch;
        K.page_stride = J.page_stride;
        K.pieces = FastDiv(J.row_bytes / 16);
        K.page_rows = FastDiv(J.page_rows);
        K.slot_end = static_cast<uint32_t>(J.num_pages * J.page_rows);
        K.row_bytes = J.row_bytes;
        A.start[A.num_jobs + 1] = A.start[A.num_jobs] + J.num_rows * K.pieces.d;
        ++A.num_jobs;
    }
    if (A.num_jobs == 0) return CSA_OK;
    int sms = 0;
    csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    if (prepare_kernel<append_kernel>(0) != cudaSuccess) return CSA_ERR_CUDA;
    const int64_t per_cta = kAppendThreads * kAppendPer;
    int64_t grid = (A.start[A.num_jobs] + per_cta - 1) / per_cta;
    if (grid > 8 * sms) grid = 8 * sms;
    return cuda_status(launch_pdl(append_kernel, dim3(static_cast<unsigned>(grid)), dim3(kAppendThreads), 0,
                                  static_cast<cudaStream_t>(stream), A, dev_status));
}

extern "C" csa_status_t csa_paged_workspace_size(const csa_paged_layout_t *layout,
                                                 const csa_params_t *params, size_t *bytes) {
    if (!bytes) return CSA_ERR_INVALID_ARGUMENT;
    csa_status_t st = check_paged(layout, params);
    if (st != CSA_OK) return st;
    *bytes = paged_attention_workspace(*layout, *params);
    return CSA_OK;
}

extern "C" csa_status_t csa_paged_attention(const csa_paged_layout_t *layout,
                                            const csa_params_t *params, const void *cache,
                                            int64_t num_pages, int64_t page_stride, const void *q,
                                            const float *sinks, csa_type_t out_type, void *out,
                                            int32_t *dev_status, void *ws, size_t ws_bytes,
                                            void *stream) {
    csa_status_t st = check_paged(layout, params);
    if (st != CSA_OK) return st;
    const csa_paged_layout_t &L = *layout;
    if (num_pages < 1 || page_stride < L.page_rows || (out_type != CSA_F32 && out_type != CSA_BF16))
        return CSA_ERR_INVALID_ARGUMENT;
    if (num_pages >= k2G || page_stride >= k2G || num_pages * page_stride >= k2G)
        return CSA_ERR_UNSUPPORTED;
    if (L.num_tokens == 0) return CSA_OK;
    if (!L.tok_seq || !L.tok_pos || !L.row_len || !L.table || !cache || !q || !out || !dev_status)
        return CSA_ERR_INVALID_ARGUMENT;
    if (!aligned(cache, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(L.tok_seq, 4) ||
        !aligned(L.tok_pos, 8) || !aligned(L.row_len, 8) || !aligned(L.table, 4) ||
        (sinks && !aligned(sinks, 4)) || !aligned(dev_status, 4))
        return CSA_ERR_INVALID_ARGUMENT;
    if (params->window > 0) {
        if (!L.swa_kv || !L.swa_first_pos || !aligned(L.swa_kv, 16) || !aligned(L.swa_first_pos, 8))
            return CSA_ERR_INVALID_ARGUMENT;
        if (L.swa_cap < params->window) return CSA_ERR_CAPACITY;
        if (static_cast<int64_t>(L.num_seqs) * L.swa_cap >= k2G) return CSA_ERR_UNSUPPORTED;
    }
    const size_t want = paged_attention_workspace(L, *params);
    if (want > 0 && (!ws || ws_bytes < want)) return CSA_ERR_WORKSPACE;
    if (ws && !aligned(ws, 256)) return CSA_ERR_INVALID_ARGUMENT;
    // several CTAs read a token's query, each at its own time, and write their
    // columns of the output
    const int64_t T = L.num_tokens, B = L.num_seqs, W = params->window > 0 ? 1 : 0;
    const int64_t vals = T * params->n_heads * kHD;
    const Range arrays[] = {{out, vals * (out_type == CSA_BF16 ? 2 : 4)}, {ws, static_cast<int64_t>(want)},
                            {dev_status, 4}, {q, vals * 2}, {sinks, int64_t(4) * params->n_heads},
                            {L.tok_seq, T * 4}, {L.tok_pos, T * 8}, {L.row_len, B * 8},
                            {L.table, B * L.max_pages * 4}, {L.swa_kv, W * B * L.swa_cap * kHD * 2},
                            {L.swa_first_pos, W * B * 8}};
    if (overlapping(arrays, 3)) return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    st = current_device(&sms);
    if (st != CSA_OK) return st;
    Launch lc{static_cast<cudaStream_t>(stream), sms};
    return cuda_status(launch_paged_attention(lc, L, *params, cache, num_pages, page_stride, q, sinks,
                                              out_type, out, dev_status, ws));
}
