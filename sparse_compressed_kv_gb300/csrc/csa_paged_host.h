// csa_paged_host.h -- argument checks that the entry points of the paged caches
// share (csa_paged.cu, csa_paged_fp8.cu).
#pragma once

#include <math.h>

#include "csa_device.cuh"
#include "csa_internal.h"

namespace csa {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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

inline csa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

inline csa_status_t check_paged(const csa_paged_layout_t *L, const csa_params_t *p) {
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

}  // namespace csa
