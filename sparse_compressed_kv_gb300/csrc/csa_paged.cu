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
// taken, pages given back) fix everything; after them every output element is
// computed by itself: token i belongs to the request whose token range holds
// i, found by bisection.  Every CTA makes the sums for itself from the 12
// bytes per request (no exchange between CTAs), keeps them in shared memory
// and writes its share of the outputs.
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxSeqs = 8192;
constexpr int64_t kPlanMaxLen = int64_t(1) << 48;

struct Req {
    int64_t len, end, old_rows, rows;
    int64_t old_pages, pages;
    int32_t add;      // new tokens
    bool over;
};

__device__ __forceinline__ Req plan_request(const csa_page_plan_t &P, int b) {
    Req r;
    r.len = P.seq_len[b];
    const int32_t nl = P.new_len[b];
    r.over = nl < 0;
    r.add = nl > 0 ? nl : 0;
    r.end = r.over ? 0 : r.len + r.add;
    r.old_rows = r.len / P.ratio;
    r.rows = r.end / P.ratio;
    r.old_pages = (r.old_rows + P.page_rows - 1) / P.page_rows;
    r.pages = (r.rows + P.page_rows - 1) / P.page_rows;
    return r;
}

struct Sums {
    int64_t tok, row, need, rel;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return {a.tok + b.tok, a.row + b.row, a.need + b.need, a.rel + b.rel};
}

__device__ __forceinline__ Sums plan_sums(const Req &r) {
    if (r.over) return {0, 0, 0, r.old_pages};
    return {r.add, r.rows - r.old_rows, r.pages - r.old_pages, 0};
}

// The last request whose range starts at or before i (ranges of requests
// without elements are empty, so the last one that starts there holds i).
__device__ __forceinline__ int plan_find(const int32_t *off, int n, int32_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const csa_page_plan_t P,
                                                                 int32_t *status) {
    extern __shared__ int32_t sm[];
    const int B = P.num_seqs;
    int32_t *tok_off = sm, *row_off = sm + B, *need_off = sm + 2 * B, *rel_off = sm + 3 * B;
    __shared__ Sums warp_sum[kPlanThreads / 32];
    __shared__ int bad_all;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad_all = 0;
    __syncthreads();

    // this thread's contiguous run of requests
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    Sums mine{0, 0, 0, 0};
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t len = P.seq_len[b];
        const int32_t nl = P.new_len[b];
        if (len < 0 || len >= kPlanMaxLen || nl < -1) {
            bad |= CSA_DEV_BAD_LENGTH;
            continue;
        }
        const Req r = plan_request(P, b);
        if (r.old_pages > P.max_pages || r.pages > P.max_pages) bad |= CSA_DEV_CAPACITY;
        mine = mine + plan_sums(r);
    }
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        Sums v;
        v.tok = __shfl_up_sync(0xffffffffu, incl.tok, o);
        v.row = __shfl_up_sync(0xffffffffu, incl.row, o);
        v.need = __shfl_up_sync(0xffffffffu, incl.need, o);
        v.rel = __shfl_up_sync(0xffffffffu, incl.rel, o);
        if (lane >= o) incl = incl + v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    if (bad) atomicOr(&bad_all, bad);
    __syncthreads();
    Sums base{0, 0, 0, 0}, total{0, 0, 0, 0};
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) base = total;
        total = total + warp_sum[w];
    }
    bad = bad_all;
    const int64_t head = P.free_pos[0], tail = P.free_pos[1], N = P.num_pages;
    if (head < 0 || tail < head || tail - head > N || tail >= kPlanMaxLen) bad |= CSA_DEV_BAD_LAYOUT;
    else if (total.need > tail - head) bad |= CSA_DEV_CAPACITY;
    else if (tail + total.rel - head > N) bad |= CSA_DEV_BAD_LAYOUT;   // more pages than the pool has
    if (total.tok > P.tok_cap || total.row > P.row_cap) bad |= CSA_DEV_CAPACITY;
    const bool ok = bad == 0;
    if (blockIdx.x == 0 && tid == 0) raise_status(status, bad);

    // exclusive offsets; a step that is refused has no tokens, blocks or pages
    Sums at{base.tok + incl.tok - mine.tok, base.row + incl.row - mine.row,
            base.need + incl.need - mine.need, base.rel + incl.rel - mine.rel};
    for (int b = b0; b < b1; ++b) {
        tok_off[b] = ok ? static_cast<int32_t>(at.tok) : 0;
        row_off[b] = ok ? static_cast<int32_t>(at.row) : 0;
        need_off[b] = ok ? static_cast<int32_t>(at.need) : 0;
        rel_off[b] = ok ? static_cast<int32_t>(at.rel) : 0;
        if (ok) at = at + plan_sums(plan_request(P, b));
    }
    if (!ok) total = Sums{0, 0, 0, 0};
    __syncthreads();

    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
    for (int64_t b = first; b <= B; b += step) {
        P.tok_off[b] = b < B ? tok_off[b] : total.tok;
        P.row_off[b] = b < B ? row_off[b] : total.row;
        if (b == B) break;
        const int64_t len = P.seq_len[b];
        const int64_t end = ok ? plan_request(P, b).end : len;
        P.seq_len_out[b] = end;
        P.row_len[b] = end > 0 ? end / P.ratio : 0;
        P.swa_first_pos[b] = end > P.swa_cap ? end - P.swa_cap : 0;
    }
    if (first < 2) P.free_pos_out[first] = first == 0 ? head + total.need : tail + total.rel;
    for (int64_t i = first; i < P.tok_cap; i += step) {
        int b = -1;
        int64_t pos = -1, slot = -1;
        if (i < total.tok) {
            b = plan_find(tok_off, B, static_cast<int32_t>(i));
            const Req r = plan_request(P, b);
            pos = r.len + (i - tok_off[b]);
            if (pos >= r.end - P.swa_cap) slot = static_cast<int64_t>(b) * P.swa_cap + pos % P.swa_cap;
        }
        P.tok_seq[i] = b;
        P.tok_pos[i] = pos;
        P.swa_slot[i] = slot;
    }
    for (int64_t i = first; i < P.row_cap; i += step) {
        int64_t slot = -1;
        if (i < total.row) {
            const int b = plan_find(row_off, B, static_cast<int32_t>(i));
            const Req r = plan_request(P, b);
            const int64_t g = r.old_rows + (i - row_off[b]);
            const int64_t pg = g / P.page_rows;
            const int32_t page = pg < r.old_pages
                                     ? P.table[static_cast<int64_t>(b) * P.max_pages + pg]
                                     : P.free_ring[(head + need_off[b] + (pg - r.old_pages)) % N];
            slot = static_cast<int64_t>(page) * P.page_rows + g % P.page_rows;
        }
        P.row_slot[i] = slot;
    }
    for (int64_t i = first; i < total.need; i += step) {
        const int b = plan_find(need_off, B, static_cast<int32_t>(i));
        const int64_t pg = plan_request(P, b).old_pages + (i - need_off[b]);
        P.table[static_cast<int64_t>(b) * P.max_pages + pg] = P.free_ring[(head + i) % N];
    }
    for (int64_t i = first; i < total.rel; i += step) {
        const int b = plan_find(rel_off, B, static_cast<int32_t>(i));
        P.free_ring[(tail + i) % N] = P.table[static_cast<int64_t>(b) * P.max_pages + (i - rel_off[b])];
    }
}

// ---------------------------------------------------------------- append

struct AppendArgs {
    csa_append_job_t job[CSA_MAX_APPEND_JOBS];
    int32_t num_jobs;
};

constexpr int kAppendThreads = 256;

// One thread per 16 bytes, grid-stride over each pair's pieces.
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs A, int32_t *status) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kAppendThreads;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
    for (int j = 0; j < A.num_jobs; ++j) {
        const csa_append_job_t &J = A.job[j];
        const int64_t pieces = J.row_bytes / 16;
        for (int64_t i = first; i < J.num_rows * pieces; i += step) {
            const int64_t row = i / pieces, c = i % pieces;
            const int64_t slot = J.slots[row];
            if (slot < 0) continue;
            if (slot >= J.num_pages * J.page_rows) {
                raise_status(status, CSA_DEV_BAD_INDEX);
                continue;
            }
            const int64_t at = slot / J.page_rows * J.page_stride + slot % J.page_rows;
            const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const char *>(J.rows) +
                                                             row * J.row_pitch + c * 16);
            *reinterpret_cast<uint4 *>(static_cast<char *>(J.cache) + at * J.row_bytes + c * 16) = v;
        }
    }
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t k2G = int64_t(1) << 31;

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
    // every CTA reads the inputs while others write the outputs
    if (P.seq_len_out == P.seq_len || P.row_len == P.seq_len || P.free_pos_out == P.free_pos)
        return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    const size_t smem = static_cast<size_t>(P.num_seqs) * 16;
    if (set_kernel_smem(page_plan_kernel, smem) != cudaSuccess) return CSA_ERR_CUDA;
    int64_t items = P.tok_cap > P.row_cap ? P.tok_cap : P.row_cap;
    if (P.num_seqs > items) items = P.num_seqs;
    int64_t grid = (items + kPlanThreads - 1) / kPlanThreads;
    if (grid > sms) grid = sms;
    page_plan_kernel<<<static_cast<unsigned>(grid), kPlanThreads, smem,
                       static_cast<cudaStream_t>(stream)>>>(P, dev_status);
    return cuda_status(cudaGetLastError());
}

extern "C" csa_status_t csa_paged_append(const csa_append_job_t *jobs, int32_t num_jobs,
                                         int32_t *dev_status, void *stream) {
    if (!jobs || num_jobs < 1 || !dev_status) return CSA_ERR_INVALID_ARGUMENT;
    if (num_jobs > CSA_MAX_APPEND_JOBS) return CSA_ERR_UNSUPPORTED;
    AppendArgs A{};
    int64_t pieces = 0;
    for (int j = 0; j < num_jobs; ++j) {
        const csa_append_job_t &J = jobs[j];
        if (J.num_rows < 0 || J.row_bytes < 16 || J.row_bytes % 16 || J.page_rows < 1 ||
            J.num_pages < 1 || J.page_stride < J.page_rows || J.row_pitch < J.row_bytes ||
            J.row_pitch % 16)
            return CSA_ERR_INVALID_ARGUMENT;
        if (J.num_pages >= k2G || J.num_pages * J.page_rows >= k2G || J.row_bytes > 65536 ||
            J.page_stride >= k2G || J.num_rows >= k2G)
            return CSA_ERR_UNSUPPORTED;
        if (J.num_rows == 0) continue;
        if (!J.rows || !J.slots || !J.cache) return CSA_ERR_INVALID_ARGUMENT;
        if (!aligned(J.rows, 16) || !aligned(J.cache, 16) || !aligned(J.slots, 8))
            return CSA_ERR_INVALID_ARGUMENT;
        A.job[A.num_jobs++] = J;
        pieces += J.num_rows * (J.row_bytes / 16);
    }
    if (A.num_jobs == 0) return CSA_OK;
    int sms = 0;
    csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    int64_t grid = (pieces + kAppendThreads - 1) / kAppendThreads;
    if (grid > 8 * sms) grid = 8 * sms;
    append_kernel<<<static_cast<unsigned>(grid), kAppendThreads, 0,
                    static_cast<cudaStream_t>(stream)>>>(A, dev_status);
    return cuda_status(cudaGetLastError());
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
    int sms = 0;
    st = current_device(&sms);
    if (st != CSA_OK) return st;
    Launch lc{static_cast<cudaStream_t>(stream), sms};
    return cuda_status(launch_paged_attention(lc, L, *params, cache, num_pages, page_stride, q, sinks,
                                              out_type, out, dev_status, ws));
}
