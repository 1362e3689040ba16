// csa_paged_fp8.cu -- 8-bit paged caches: the C entry points, the quantising
// append and the read (include/csa.h, "8-bit paged caches").  The attention
// over the pages is in csa_paged_attention_fp8.cu.
#include "csa_fp8.cuh"
#include "csa_paged_host.h"

namespace csa {
namespace {

constexpr int kFp8MaxWidth = 1024;
constexpr int kFp8Threads = 256;
constexpr int kFp8Warps = kFp8Threads / 32;

// ---------------------------------------------------------------- append

struct AppendFp8Job {
    const char *rows;
    const int64_t *slots;
    uint8_t *cache;
    float *scales;
    int64_t row_pitch, page_stride, scale_stride;
    FastDiv page_rows;
    uint32_t slot_end, units;                          // units: 8 values each, of a row
    int32_t f32;
};
struct AppendFp8Args {
    AppendFp8Job job[CSA_MAX_APPEND_JOBS];
    int64_t start[CSA_MAX_APPEND_JOBS + 1];            // first row of each pair, all of them
    int32_t num_jobs;
};

// The scale's exponent from the bits of a row's largest finite magnitude, 1.m 2^e:
// it is at most 1.75 2^(8 + k) where k = e - 8 and m <= .75, else k = e - 7.
__device__ __forceinline__ int fp8_exponent(uint32_t amax) {
    const int k = static_cast<int>(amax >> 23) - (127 + 8) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(k, -kFp8MaxExp), kFp8MaxExp);
}

constexpr uint32_t kFp8Largest = (60u + 8 + 127) << 23 | 0x600000u;   // 448 * 2^60, as f32 bits

// Eight values of a row, bf16 or f32.
struct Values {
    float x[8];
    __device__ __forceinline__ Values(const uint4 (&raw)[2], bool f32) {
        const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = __uint_as_float(f32 ? w[e] : e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
};

// One warp a row: its values stay in registers between the maximum and the
// codes, so a row is read once; a lane has up to kUnits runs of 8 values.  kRows rows at a
// time, and the slots of the next ones on their way, keep bytes in flight, and CTAs that
// stay (8 per SM) walk on without a start of their own.  Two caches, 163,840 bf16 rows of
// 512 values of which 120,136 have a slot (the rings keep the newest ones): 41.4 us, 4.5
// TB/s of the 186 MB that move (the copy's rate: 27.4 us); rows without a slot take their
// turns all the same.  120,136 rows that all have one, at random: 37.8 us, 4.9 TB/s, from
// f32 56.3 us, 5.5.  So DRAM is not what bounds it; what does was not found out.  One row
// at a time took 50.6, three 54.8 (fewer CTAs fit), two with 4 and 16 CTAs per SM 42.3 and
// 41.4.  40 rows: 1.9 us, a launch and two trips to memory.  Rows above 512 values take one
// at a time (twice the registers).
template <int kUnits, int kRows>
__global__ void __launch_bounds__(kFp8Threads) append_fp8_kernel(const AppendFp8Args A, int32_t *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t all = A.start[A.num_jobs], step = static_cast<int64_t>(gridDim.x) * kFp8Warps;
    auto job_of = [&](int64_t i) {
        int j = 0;
#pragma unroll
        for (int q = 1; q < CSA_MAX_APPEND_JOBS; ++q)
            if (q < A.num_jobs && i >= A.start[q]) j = q;
        return j;
    };
    auto slot_of = [&](int64_t i) {
        if (i >= all) return int64_t(-1);
        const int j = job_of(i);
        return A.job[j].slots[i - A.start[j]];
    };
    int bad = 0;
    int64_t i0 = static_cast<int64_t>(blockIdx.x) * kFp8Warps + (threadIdx.x >> 5);
    int64_t coming[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) coming[r] = slot_of(i0 + r * step);
    for (; i0 < all; i0 += kRows * step) {
        int64_t slot[kRows];
        uint4 raw[kRows][kUnits][2];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t i = i0 + r * step;
            const int j = job_of(i);
            const AppendFp8Job &J = A.job[j];
            slot[r] = coming[r];
            if (slot[r] >= J.slot_end) {
                bad = CSA_DEV_BAD_INDEX;
                slot[r] = -1;
            }
            const char *const src = J.rows + (i - A.start[j]) * J.row_pitch;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const uint32_t at = lane + 32 * u;
                raw[r][u][0] = raw[r][u][1] = make_uint4(0, 0, 0, 0);
                if (slot[r] < 0 || at >= J.units) continue;
                if (J.f32) {
                    raw[r][u][0] = __ldcs(reinterpret_cast<const uint4 *>(src + at * 32));
                    raw[r][u][1] = __ldcs(reinterpret_cast<const uint4 *>(src + at * 32 + 16));
                } else {
                    raw[r][u][0] = __ldcs(reinterpret_cast<const uint4 *>(src + at * 16));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) coming[r] = slot_of(i0 + (kRows + r) * step);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (slot[r] < 0) continue;
            const AppendFp8Job &J = A.job[job_of(i0 + r * step)];
            // the largest magnitude, of two numbers at a time for bf16
            uint32_t amax = 0;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const uint4 a = raw[r][u][0], b = raw[r][u][1];
                if (J.f32) {
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) amax = max(amax, w[e] & 0x7FFFFFFFu);
                } else {
                    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu),
                                                __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
                    amax = max(amax, max(m << 16, m & 0xFFFF0000u));
                }
            }
            amax = __reduce_max_sync(0xffffffffu, amax);
            // something infinite, NaN or above the largest scale: these become NaN, and the
            // scale is that of the others
            const bool odd = amax > kFp8Largest;
            if (odd) {
                uint32_t m = 0;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const Values v(raw[r][u], J.f32);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t x = __float_as_uint(v.x[e]) & 0x7FFFFFFFu;
                        m = max(m, x < 0x7F800000u ? x : 0u);
                    }
                }
                amax = __reduce_max_sync(0xffffffffu, m);
            }
            const int k = fp8_exponent(amax);
            const float inv = exponent_f32(-k);
            const uint32_t s = static_cast<uint32_t>(slot[r]), page = J.page_rows.div(s), in = s - page * J.page_rows.d;
            uint8_t *const dst = J.cache + (page * J.page_stride + in) * (J.units * 8);
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const uint32_t at = lane + 32 * u;
                if (at >= J.units) break;
                Values y(raw[r][u], J.f32);
#pragma unroll
                for (int e = 0; e < 8; ++e) y.x[e] *= inv;
                if (odd) {                               // (the conversion would saturate)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!(fabsf(y.x[e]) <= 448.f)) y.x[e] = NAN;
                }
                *reinterpret_cast<uint2 *>(dst + at * 8) =
                    make_uint2(e4m3x4(y.x[0], y.x[1], y.x[2], y.x[3]), e4m3x4(y.x[4], y.x[5], y.x[6], y.x[7]));
            }
            if (lane == 0) J.scales[page * J.scale_stride + in] = exponent_f32(k);
        }
    }
    if (lane == 0) raise_status(status, bad);
}

// ---------------------------------------------------------------- read

struct ReadFp8Args {
    csa_read_fp8_t R;
    FastDiv page_rows;
    uint32_t slot_end;
};

// One warp a row, 16 bytes of the output a lane at a time, two ahead of the first
// store, and the slot of the next row.  Bound by the bytes: 131,072 rows of 512 values to
// f32 take 54.9 us, 6.1 TB/s (the copy's rate: 49.7 us), with up to 64 CTAs' worth of rows
// per SM; 16: 55.3; a thread for 16 bytes, without the slots ahead: 65.6.
template <bool kF32>
__global__ void __launch_bounds__(kFp8Threads) read_fp8_kernel(const ReadFp8Args A, int32_t *status) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kVals = kF32 ? 4 : 8;
    const csa_read_fp8_t &R = A.R;
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kFp8Warps;
    int bad = 0;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kFp8Warps + (threadIdx.x >> 5);
    int64_t coming = i < R.num_rows ? R.slots[i] : -1;
    for (; i < R.num_rows; i += step) {
        const int64_t slot = coming;
        coming = i + step < R.num_rows ? R.slots[i + step] : -1;
        if (slot < 0) continue;
        if (slot >= A.slot_end) {
            bad = CSA_DEV_BAD_INDEX;
            continue;
        }
        const uint32_t s = static_cast<uint32_t>(slot), page = A.page_rows.div(s), in = s - page * A.page_rows.d;
        const uint8_t *const src = static_cast<const uint8_t *>(R.cache) + (page * R.page_stride + in) * R.width;
        const float scale = R.scales[page * R.scale_stride + in];
        char *const dst = static_cast<char *>(R.out) + i * R.out_pitch;
        const int pieces = R.width / kVals;
        for (int c = lane; c < pieces; c += 64) {
            uint2 w[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                w[u] = make_uint2(0, 0);
                if (c + 32 * u >= pieces) continue;
                if (kF32) w[u].x = *reinterpret_cast<const uint32_t *>(src + (c + 32 * u) * 4);
                else w[u] = *reinterpret_cast<const uint2 *>(src + (c + 32 * u) * 8);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (c + 32 * u >= pieces) continue;
                float v[8];
                e4m3x4_values(w[u].x, v);
                if (!kF32) e4m3x4_values(w[u].y, v + 4);
#pragma unroll
                for (int e = 0; e < kVals; ++e) v[e] *= scale;
                *reinterpret_cast<uint4 *>(dst + (c + 32 * u) * 16) =
                    kF32 ? make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]))
                         : make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                      pack_bf16x2(v[6], v[7]));
            }
        }
    }
    if (lane == 0) raise_status(status, bad);
}

bool bad_pool(int32_t width, int32_t page_rows, int64_t num_pages, int64_t page_stride, int64_t scale_stride) {
    return width < 16 || width % 16 || page_rows < 1 || num_pages < 1 || page_stride < page_rows ||
           scale_stride < page_rows;
}

bool large_pool(int32_t width, int32_t page_rows, int64_t num_pages, int64_t page_stride, int64_t scale_stride) {
    return width > kFp8MaxWidth || num_pages >= k2G || num_pages * page_rows >= k2G || page_stride >= k2G ||
           scale_stride >= k2G;
}

// the bytes from a pool's first row to its last (what lies behind the last page's
// rows belongs to others)
int64_t pool_bytes(int64_t num_pages, int64_t stride, int32_t page_rows, int64_t row_bytes) {
    return ((num_pages - 1) * stride + page_rows) * row_bytes;
}

bool shared(const Range &a, const Range &b) {
    const Range r[2] = {a, b};
    return overlapping(r, 1);
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_paged_append_fp8(const csa_append_fp8_job_t *jobs, int32_t num_jobs,
                                             int32_t *dev_status, void *stream) {
    if (!jobs || num_jobs < 1 || !dev_status || !aligned(dev_status, 4)) return CSA_ERR_INVALID_ARGUMENT;
    if (num_jobs > CSA_MAX_APPEND_JOBS) return CSA_ERR_UNSUPPORTED;
    AppendFp8Args A{};
    Range given[2 * CSA_MAX_APPEND_JOBS + 1], written[2 * CSA_MAX_APPEND_JOBS];
    uint32_t most = 0;
    for (int j = 0; j < num_jobs; ++j) {
        const csa_append_fp8_job_t &J = jobs[j];
        if (J.type != CSA_F32 && J.type != CSA_BF16) return CSA_ERR_INVALID_ARGUMENT;
        const int64_t row_bytes = static_cast<int64_t>(J.width) * (J.type == CSA_F32 ? 4 : 2);
        if (J.num_rows < 0 || bad_pool(J.width, J.page_rows, J.num_pages, J.page_stride, J.scale_stride) ||
            J.row_pitch < row_bytes || J.row_pitch % 16)
            return CSA_ERR_INVALID_ARGUMENT;
        if (large_pool(J.width, J.page_rows, J.num_pages, J.page_stride, J.scale_stride) || J.num_rows >= k2G ||
            J.row_pitch >= k2G)
            return CSA_ERR_UNSUPPORTED;
        if (J.num_rows == 0) continue;
        if (!J.rows || !J.slots || !J.cache || !J.scales) return CSA_ERR_INVALID_ARGUMENT;
        if (!aligned(J.rows, 16) || !aligned(J.cache, 16) || !aligned(J.slots, 8) || !aligned(J.scales, 4))
            return CSA_ERR_INVALID_ARGUMENT;
        const int n = A.num_jobs;
        AppendFp8Job &K = A.job[n];
        K.rows = static_cast<const char *>(J.rows);
        K.slots = J.slots;
        K.cache = static_cast<uint8_t *>(J.cache);
        K.scales = J.scales;
        K.row_pitch = J.row_pitch;
        K.page_stride = J.page_stride;
        K.scale_stride = J.scale_stride;
        K.page_rows = FastDiv(J.page_rows);
        K.slot_end = static_cast<uint32_t>(J.num_pages * J.page_rows);
        K.units = J.width / 8;
        K.f32 = J.type == CSA_F32;
        given[2 * n] = {J.rows, (J.num_rows - 1) * J.row_pitch + row_bytes};
        given[2 * n + 1] = {J.slots, J.num_rows * 8};
        written[2 * n] = {J.cache, pool_bytes(J.num_pages, J.page_stride, J.page_rows, J.width)};
        written[2 * n + 1] = {J.scales, pool_bytes(J.num_pages, J.scale_stride, J.page_rows, 4)};
        if (K.units > most) most = K.units;
        A.start[n + 1] = A.start[n] + J.num_rows;
        ++A.num_jobs;
    }
    if (A.num_jobs == 0) return CSA_OK;
    given[2 * A.num_jobs] = {dev_status, 4};
    for (int w = 0; w < 2 * A.num_jobs; ++w)
        for (int g = 0; g <= 2 * A.num_jobs; ++g)
            if (shared(written[w], given[g])) return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    const csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    int64_t grid = (A.start[A.num_jobs] + kFp8Warps - 1) / kFp8Warps;
    if (grid > 8 * sms) grid = 8 * sms;
    const dim3 g(static_cast<unsigned>(grid)), b(kFp8Threads);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto units) {
        constexpr int kUnits = decltype(units)::value;
        constexpr auto kernel = append_fp8_kernel<kUnits, kUnits == 4 ? 1 : 2>;
        const cudaError_t e = prepare_kernel<kernel>(0);
        return cuda_status(e != cudaSuccess ? e : launch_pdl(kernel, g, b, 0, s, A, dev_status));
    };
    if (most <= 32) return launch(std::integral_constant<int, 1>{});
    if (most <= 64) return launch(std::integral_constant<int, 2>{});
    return launch(std::integral_constant<int, 4>{});
}

extern "C" csa_status_t csa_paged_read_fp8(const csa_read_fp8_t *read, int32_t *dev_status, void *stream) {
    if (!read || !dev_status || !aligned(dev_status, 4)) return CSA_ERR_INVALID_ARGUMENT;
    const csa_read_fp8_t &R = *read;
    if (R.type != CSA_F32 && R.type != CSA_BF16) return CSA_ERR_INVALID_ARGUMENT;
    const int64_t row_bytes = static_cast<int64_t>(R.width) * (R.type == CSA_F32 ? 4 : 2);
    if (R.num_rows < 0 || bad_pool(R.width, R.page_rows, R.num_pages, R.page_stride, R.scale_stride) ||
        R.out_pitch < row_bytes || R.out_pitch % 16)
        return CSA_ERR_INVALID_ARGUMENT;
    if (large_pool(R.width, R.page_rows, R.num_pages, R.page_stride, R.scale_stride) || R.num_rows >= k2G ||
        R.out_pitch >= k2G)
        return CSA_ERR_UNSUPPORTED;
    if (R.num_rows == 0) return CSA_OK;
    if (!R.cache || !R.scales || !R.slots || !R.out) return CSA_ERR_INVALID_ARGUMENT;
    if (!aligned(R.cache, 16) || !aligned(R.scales, 4) || !aligned(R.slots, 8) || !aligned(R.out, 16))
        return CSA_ERR_INVALID_ARGUMENT;
    const Range arrays[] = {{R.out, (R.num_rows - 1) * R.out_pitch + row_bytes}, {dev_status, 4},
                            {R.slots, R.num_rows * 8},
                            {R.cache, pool_bytes(R.num_pages, R.page_stride, R.page_rows, R.width)},
                            {R.scales, pool_bytes(R.num_pages, R.scale_stride, R.page_rows, 4)}};
    if (overlapping(arrays, 2)) return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    const csa_status_t st = current_device(&sms);
    if (st != CSA_OK) return st;
    int64_t grid = (R.num_rows + kFp8Warps - 1) / kFp8Warps;
    if (grid > 64 * sms) grid = 64 * sms;
    const ReadFp8Args A{R, FastDiv(R.page_rows), static_cast<uint32_t>(R.num_pages * R.page_rows)};
    const dim3 g(static_cast<unsigned>(grid)), b(kFp8Threads);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto f32) {
        constexpr auto kernel = read_fp8_kernel<decltype(f32)::value>;
        const cudaError_t e = prepare_kernel<kernel>(0);
        return cuda_status(e != cudaSuccess ? e : launch_pdl(kernel, g, b, 0, s, A, dev_status));
    };
    return R.type == CSA_F32 ? launch(std::true_type{}) : launch(std::false_type{});
}

extern "C" csa_status_t csa_paged_attention_fp8(const csa_paged_layout_t *layout, const csa_params_t *params,
                                                const void *cache, const float *scales,
                                                const float *swa_scales, int64_t num_pages,
                                                int64_t page_stride, int64_t scale_stride, const void *q,
                                                const float *sinks, csa_type_t out_type, void *out,
                                                int32_t *dev_status, void *ws, size_t ws_bytes,
                                                void *stream) {
    csa_status_t st = check_paged(layout, params);
    if (st != CSA_OK) return st;
    const csa_paged_layout_t &L = *layout;
    if (num_pages < 1 || page_stride < L.page_rows || scale_stride < L.page_rows ||
        (out_type != CSA_F32 && out_type != CSA_BF16))
        return CSA_ERR_INVALID_ARGUMENT;
    if (num_pages >= k2G || page_stride >= k2G || scale_stride >= k2G || num_pages * page_stride >= k2G)
        return CSA_ERR_UNSUPPORTED;
    if (L.num_tokens == 0) return CSA_OK;
    if (!L.tok_seq || !L.tok_pos || !L.row_len || !L.table || !cache || !scales || !q || !out || !dev_status)
        return CSA_ERR_INVALID_ARGUMENT;
    if (!aligned(cache, 16) || !aligned(scales, 4) || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(L.tok_seq, 4) || !aligned(L.tok_pos, 8) || !aligned(L.row_len, 8) || !aligned(L.table, 4) ||
        (sinks && !aligned(sinks, 4)) || !aligned(dev_status, 4))
        return CSA_ERR_INVALID_ARGUMENT;
    if (params->window > 0) {
        if (!L.swa_kv || !swa_scales || !L.swa_first_pos || !aligned(L.swa_kv, 16) || !aligned(swa_scales, 4) ||
            !aligned(L.swa_first_pos, 8))
            return CSA_ERR_INVALID_ARGUMENT;
        if (L.swa_cap < params->window) return CSA_ERR_CAPACITY;
        if (static_cast<int64_t>(L.num_seqs) * L.swa_cap >= k2G) return CSA_ERR_UNSUPPORTED;
    }
    const size_t want = paged_attention_workspace(L, *params);
    if (!ws || ws_bytes < want) return CSA_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return CSA_ERR_INVALID_ARGUMENT;
    // several CTAs read a token's query, each at its own time, and write their
    // columns of the output
    const int64_t T = L.num_tokens, B = L.num_seqs, W = params->window > 0 ? 1 : 0;
    const int64_t vals = T * params->n_heads * kHD;
    const Range arrays[] = {{out, vals * (out_type == CSA_BF16 ? 2 : 4)}, {ws, static_cast<int64_t>(want)},
                            {dev_status, 4}, {q, vals * 2}, {sinks, int64_t(4) * params->n_heads},
                            {L.tok_seq, T * 4}, {L.tok_pos, T * 8}, {L.row_len, B * 8},
                            {L.table, B * L.max_pages * 4}, {L.swa_kv, W * B * L.swa_cap * kHD},
                            {swa_scales, W * B * L.swa_cap * 4}, {L.swa_first_pos, W * B * 8}};
    if (overlapping(arrays, 3)) return CSA_ERR_INVALID_ARGUMENT;
    int sms = 0;
    st = current_device(&sms);
    if (st != CSA_OK) return st;
    const Launch lc{static_cast<cudaStream_t>(stream), sms};
    return cuda_status(launch_paged_attention_fp8(lc, L, *params, cache, scales, swa_scales, num_pages,
                                                  page_stride, scale_stride, q, sinks, out_type, out,
                                                  dev_status, ws));
}
