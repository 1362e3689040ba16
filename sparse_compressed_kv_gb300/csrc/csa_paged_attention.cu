// csa_paged_attention.cu -- shared-KV attention of new tokens over a paged
// cache and the window ring:
//   l_j = scale q_h . row_j,   out_h = sum_j softmax_j(l [, sink]) row_j.
// One CTA per (token, head) walks the token's rows: each warp takes a row's
// logit, then every thread accumulates two of the 512 output columns.
#include <math.h>

#include "csa_device.cuh"
#include "csa_internal.h"

namespace csa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;   // rows per softmax step

struct PagedArgs {
    csa_paged_layout_t L;
    int32_t H, window, ratio;
    float scale;
    const __nv_bfloat16 *cache;
    int64_t num_pages, page_stride;
    const __nv_bfloat16 *q;
    const float *sinks;
    void *out;
    int32_t bf16_out;
    int32_t *status;
};

__global__ void __launch_bounds__(kThreads) paged_attention_kernel(const PagedArgs A) {
    const int h = blockIdx.x, t = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = A.L.tok_seq[t];
    if (b == -1) return;
    __shared__ const __nv_bfloat16 *row[kTile];
    __shared__ float logit[kTile];
    const int64_t pos = A.L.tok_pos[t];
    int bad = 0;
    int64_t n = 0, first = 0, near = 0;
    if (b < 0 || b >= A.L.num_seqs || pos < 0) {
        bad = CSA_DEV_BAD_LAYOUT;
    } else {
        n = A.L.row_len[b];
        const int64_t cap = static_cast<int64_t>(A.L.max_pages) * A.L.page_rows;
        if (n < 0) bad |= CSA_DEV_BAD_LENGTH, n = 0;
        if (n > cap) bad |= CSA_DEV_CAPACITY, n = cap;
        if (pos / A.ratio < n) n = pos / A.ratio;
        first = window_first(pos, A.window);
        near = A.window > 0 ? pos - first + 1 : 0;
    }
    const __nv_bfloat16 *q = A.q + (static_cast<int64_t>(t) * A.H + h) * kHD;
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int64_t j0 = 0; j0 < n + near; j0 += kTile) {
        if (tid < kTile) {
            const int64_t j = j0 + tid;
            const __nv_bfloat16 *p = nullptr;
            if (j < n) {
                const int32_t page = A.L.table[static_cast<int64_t>(b) * A.L.max_pages + j / A.L.page_rows];
                if (page < 0 || page >= A.num_pages) bad |= CSA_DEV_BAD_INDEX;
                else p = A.cache + (page * A.page_stride + j % A.L.page_rows) * kHD;
            } else if (j < n + near) {
                const int64_t x = first + (j - n);
                if (x < A.L.swa_first_pos[b]) bad |= CSA_DEV_MISSING_SWA;
                else
                    p = static_cast<const __nv_bfloat16 *>(A.L.swa_kv) +
                        (static_cast<int64_t>(b) * A.L.swa_cap + x % A.L.swa_cap) * kHD;
            }
            row[tid] = p;
        }
        __syncthreads();
        for (int r = warp; r < kTile; r += kThreads / 32) {
            const __nv_bfloat16 *p = row[r];
            float s = 0.f;
            if (p)
                for (int d = lane; d < kHD; d += 32) s += __bfloat162float(q[d]) * __bfloat162float(p[d]);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) logit[r] = p ? s * A.scale : -INFINITY;
        }
        __syncthreads();
        float mc = m;
        for (int r = 0; r < kTile; ++r) mc = fmaxf(mc, logit[r]);
        if (mc != -INFINITY) {
            const float a = expf(m - mc);
            o0 *= a;
            o1 *= a;
            l *= a;
            m = mc;
            for (int r = 0; r < kTile; ++r) {
                const __nv_bfloat16 *p = row[r];
                if (!p) continue;
                const float w = expf(logit[r] - m);
                l += w;
                o0 += w * __bfloat162float(p[2 * tid]);
                o1 += w * __bfloat162float(p[2 * tid + 1]);
            }
        }
        __syncthreads();
    }
    raise_status(A.status, bad);
    float z = l;
    if (A.sinks && m != -INFINITY) z += expf(A.sinks[h] - m);
    const float f = l > 0.f ? 1.f / z : 0.f;
    const int64_t at = (static_cast<int64_t>(t) * A.H + h) * kHD + 2 * tid;
    if (A.bf16_out) {
        static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(o0 * f);
        static_cast<__nv_bfloat16 *>(A.out)[at + 1] = __float2bfloat16(o1 * f);
    } else {
        static_cast<float *>(A.out)[at] = o0 * f;
        static_cast<float *>(A.out)[at + 1] = o1 * f;
    }
}

}  // namespace

size_t paged_attention_workspace(const csa_paged_layout_t &, const csa_params_t &) { return 256; }

cudaError_t launch_paged_attention(const Launch &lc, const csa_paged_layout_t &L,
                                   const csa_params_t &p, const void *cache, int64_t num_pages,
                                   int64_t page_stride, const void *q, const float *sinks,
                                   csa_type_t out_type, void *out, int32_t *status, void *) {
    PagedArgs A{};
    A.L = L;
    A.H = p.n_heads;
    A.window = p.window;
    A.ratio = p.ratio;
    A.scale = p.scale;
    A.cache = static_cast<const __nv_bfloat16 *>(cache);
    A.num_pages = num_pages;
    A.page_stride = page_stride;
    A.q = static_cast<const __nv_bfloat16 *>(q);
    A.sinks = sinks;
    A.out = out;
    A.bf16_out = out_type == CSA_BF16;
    A.status = status;
    paged_attention_kernel<<<dim3(p.n_heads, L.num_tokens), kThreads, 0, lc.stream>>>(A);
    return cudaGetLastError();
}

}  // namespace csa
