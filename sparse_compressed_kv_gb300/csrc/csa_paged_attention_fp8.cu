// csa_paged_attention_fp8.cu -- shared-KV attention of new tokens over a paged
// cache of e4m3 rows and their window ring:
//   l_j = scale q_h . (s_j c_j),   out_h = sum_j softmax_j(l [, sink]) s_j c_j.
//
// One warp a token and head: a lane has 16 columns of the query, each row is
// read, its product summed over the warp, and the running sums rescaled where
// the maximum rises; every 256 rows the sums go to a second level (one sum of
// 40,000 equal terms is off by 6e-4).
#include "csa_fp8.cuh"
#include "csa_paged_attention.cuh"

namespace csa {
namespace {

struct PagedFp8Args : PagedArgs {
    const uint8_t *codes;
    const float *scales, *swa_scales;
    int64_t scale_stride;
    const __nv_bfloat16 *q;
};

constexpr int kHeadWarps = 8;

__global__ void __launch_bounds__(kHeadWarps * 32) paged_attention_fp8_kernel(const PagedFp8Args A) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, t = blockIdx.x, h = blockIdx.y * kHeadWarps + (threadIdx.x >> 5);
    int bad = 0;
    const Rec r = token_rec(A, t, max(1, A.L.num_tokens / A.L.num_seqs), bad);
    if (h >= A.H) return;
    if (r.b >= 0) {
        float q[16], acc[16], acc2[16];
        const int64_t at = (static_cast<int64_t>(t) * A.H + h) * kHD + 16 * lane;
        for (int i = 0; i < 16; ++i) {
            q[i] = __bfloat162float(A.q[at + i]);
            acc[i] = acc2[i] = 0.f;
        }
        float m = -INFINITY, l = 0.f, l2 = 0.f;
        int since = 0;
        auto add = [&](const uint8_t *row, float s) {
            const uint4 w = *reinterpret_cast<const uint4 *>(row + 16 * lane);
            float v[16], d = 0.f;
            e4m3x4_values(w.x, v);
            e4m3x4_values(w.y, v + 4);
            e4m3x4_values(w.z, v + 8);
            e4m3x4_values(w.w, v + 12);
            for (int i = 0; i < 16; ++i) {
                v[i] *= s;
                d = fmaf(q[i], v[i], d);
            }
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            d *= A.scale_log2;
            if (d > m) {
                const float f = exp2f(m - d);
                l *= f;
                l2 *= f;
                for (int i = 0; i < 16; ++i) {
                    acc[i] *= f;
                    acc2[i] *= f;
                }
                m = d;
            }
            const float p = exp2f(d - m);
            l += p;
            for (int i = 0; i < 16; ++i) acc[i] = fmaf(p, v[i], acc[i]);
            if (++since < 256) return;
            since = 0;
            l2 += l;
            l = 0.f;
            for (int i = 0; i < 16; ++i) {
                acc2[i] += acc[i];
                acc[i] = 0.f;
            }
        };
        for (int j = 0; j < r.n; ++j) {
            const int pg = A.page_div.div(j);
            const int32_t page = A.L.table[static_cast<int64_t>(r.b) * A.L.max_pages + pg];
            if (page < 0 || page >= A.num_pages) {
                bad |= CSA_DEV_BAD_INDEX;
                continue;
            }
            const int in = j - pg * A.L.page_rows;
            add(A.codes + (page * A.page_stride + in) * kHD, A.scales[page * A.scale_stride + in]);
        }
        for (int j = 0; j < r.near; ++j) {
            if (r.first + j < r.first_res) {
                bad |= CSA_DEV_MISSING_SWA;
                continue;
            }
            const int64_t i = static_cast<int64_t>(r.b) * A.L.swa_cap + A.swa_div.mod64(r.first + j);
            add(static_cast<const uint8_t *>(A.L.swa_kv) + i * kHD, A.swa_scales[i]);
        }
        l += l2;
        float z = l;
        if (A.sinks && m != -INFINITY) z += exp2f(A.sinks[h] * kLog2e - m);
        const float f = m == -INFINITY && l == 0.f ? 0.f : 1.f / z;
        for (int i = 0; i < 16; ++i) {
            const float o = (acc[i] + acc2[i]) * f;
            if (A.bf16_out) static_cast<__nv_bfloat16 *>(A.out)[at + i] = __float2bfloat16(o);
            else static_cast<float *>(A.out)[at + i] = o;
        }
    }
    if (lane == 0 && h == 0) raise_status(A.status, bad);
}

}  // namespace

cudaError_t launch_paged_attention_fp8(const Launch &lc, const csa_paged_layout_t &L,
                                       const csa_params_t &p, const void *cache, const float *scales,
                                       const float *swa_scales, int64_t num_pages,
                                       int64_t page_stride, int64_t scale_stride, const void *q,
                                       const float *sinks, csa_type_t out_type, void *out,
                                       int32_t *status, void *ws) {
    PagedFp8Args A{};
    static_cast<PagedArgs &>(A) = paged_args(lc, L, p, num_pages, page_stride, sinks, out_type, out, status, ws);
    A.codes = static_cast<const uint8_t *>(cache);
    A.scales = scales;
    A.swa_scales = swa_scales;
    A.scale_stride = scale_stride;
    A.q = static_cast<const __nv_bfloat16 *>(q);
    const cudaError_t e = prepare_kernel<paged_attention_fp8_kernel>(0);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attention_fp8_kernel, dim3(L.num_tokens, (p.n_heads + kHeadWarps - 1) / kHeadWarps),
                      dim3(kHeadWarps * 32), 0, lc.stream, A);
}

}  // namespace csa
