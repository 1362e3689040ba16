// csa_paged_attention_fp8.cu -- shared-KV attention of new tokens over a paged
// cache of e4m3 rows and their window ring, on the 5th-generation tensor cores:
//   l_j = scale q_h . (s_j c_j),   out_h = sum_j softmax_j(l [, sink]) s_j c_j.
//
// The division of the work, the segments, the partials and the joins are those
// of the bf16 rows' kernel (csa_paged_attention.cuh); a chunk is 64 row slots, and
// the codes are the tensor cores' operands as they lie in memory:
//   warps 0..7    where a segment begins, its query's heads by turns, split in two e4m3
//                 terms; softmax with a lazily raised maximum, warps 0..3 of the
//                 chunk's rows 0..31, warps 4..7 of the others;
//                 and a segment's epilogue, under the next segment's first logits
//   warp 8        S = Q . rows^T (M = 64 heads x 2 terms from tensor memory, N = 64
//                 rows, K = 512)
//   warp 9        O^T += rows^T . P^T (M = 128 columns a tile, N = 64 heads, K = 64 rows)
//   warps 10, 11  fetch a chunk's rows, 32 each: 8 rows of one page are one TMA box
//                 (128 columns x 8 rows x 4 column groups: 4 KiB), others go row by
//                 row with 16-byte cp.async; and each row's scale
// A group's 4 KiB hold 4 column groups of 8 rows x 128 bytes (the swizzle atom):
// the K-major operand of S and the MN-major operand of O^T.
//
// Q = hi + lo: a head's largest magnitude is brought to [2^7, 2^8) by a power of
// two; hi is the nearest e4m3 value, lo the nearest to what is left.  A bf16
// number has 8 bits and each term takes 4, so the two are exact down to 2^-10 of
// 2^8 (lo's last place is 2^-9; below that a value is off by up to 2^-10, 2^-17 of its
// head's largest).  Rows 32 q + i and 32 q + 16 + i of the operand are the terms of head
// 16 q + i, so that both sums lie in the same warp's quarter of tensor memory, and the
// softmax adds them.
//
// P = 2^(l_j - m) s_j as e5m2 terms of 3 bits: what f16 rounds it to (2^-11), cut into
// bytes (e5m2 is f16's upper byte), three terms for a bf16 output (2^-9), six for
// f32 (2^-18 in all).  e4m3 would hold 4 bits a term, but 18 powers of two; e5m2 holds 32:
// with the maximum m of l_j + log2 s_j brought to 2^7 (and up to 2^15 before it is
// raised) its last place is 2^-23 of the largest weight, however many terms there are.
// What a weight is off by there goes into the next one (last_bytes), so that small weights
// keep their sum.
//
// What bounds it, with 64 heads: shared memory, which passes 128 bytes a cycle.  For a
// bf16 output a chunk's products read 176 KB (the rows once for S and once a term for
// O^T, the weights once a tile), 32 KB of rows and 12 KB of weights are written: 1,720
// cycles.  (The products alone: 16 x 32 cycles for S, A in tensor memory, and 24 x 48 for
// O^T, 1,670.)  The loop takes 1,920; for an f32 output 352 KB, 2,750, and 2,960 (3,200
// where a segment goes through the partial every 27 chunks).  540,000 rows of 32 contexts
// 74.2 us (3.7 TB/s; the bytes alone 40.8), a million tokens at ratio 4 (262,144 rows) 43.6
// us (20.0).  Beside a rule below stand its two sides in this build, replayed from a graph;
// where the other side's code is gone, in the build that chose.
// Three terms of 64 columns read a tile of O^T's A three times; one product of 128
// or 192 columns would not, but the accumulators would need 512 or 768 columns of tensor
// memory.  What a call begins and ends with, one long context on all SMs: 3,000 cycles
// until the query is there, 4,200 to split and store it, 2,400 to the first O^T product;
// 4,000 for the drain of a partial (128 KiB at 32 bytes a cycle); and the join's kernel.
#include <cuda_fp16.h>

#include <type_traits>

#include "csa_fp8.cuh"
#include "csa_paged_attention.cuh"

namespace csa {
namespace {

constexpr int kThreads = 384;
constexpr int kSmThreads = 256;                 // warps 0..7, half of them for each 32 rows of a chunk
constexpr int kSmGroup = kSmThreads / 2;        // that half
constexpr int kChunk = 64;
constexpr int kSteps = kChunk / 32;             // of 32 rows: a fetch warp, half of the softmax, a K step of O^T each
constexpr int kGroupBytes = 8 * kHD;            // 8 rows: 4 KiB
constexpr int kStageBytes = kChunk / 8 * kGroupBytes;   // 32 KiB
// What shared memory has room for beside two buffers of P (12 KiB each, 24 KiB with
// an f32 output): a row takes 1,300 to 1,900 cycles from its copy's start, as long as a
// chunk's products, and a stage is held by two of them besides.
template <int kTerms>
constexpr int kStages = kTerms == 3 ? 6 : 5;
constexpr int kPBufs = 2;
constexpr int kMaxStages = 6;
constexpr int kStagedHeads = 16;                // of a bf16 output, on their way through shared memory (P's)
constexpr int kTermBytes = kHG * 16;            // 16 rows of a term of P
template <int kTerms>
constexpr int kPieceBytes = kTerms * kTermBytes;
// Tensor memory: S in buffers of 64 columns; O^T, 4 tiles of 64 columns (heads); the
// query, 128 rows x 512 codes.  With an f32 output's six terms the columns of a second S
// buffer go to the first tile, which takes two terms from one reading of its rows into 64
// columns each (128-head drafts 75.5 us, with two buffers instead 78.7; a bf16 output's
// three: 32 contexts 73.8 us and 74.2, one of 8,192 rows 14.2 either way).
template <int kTerms>
constexpr int kSBufs = kTerms == 3 ? 2 : 1;
template <int kTerms>
constexpr int kWide = kTerms == 3 ? 0 : 1;      // tiles of O^T that take two terms at a time
constexpr int kSCol = 0;
template <int kTerms>
constexpr int kOCol = 64 * kSBufs<kTerms>;
constexpr int kQCol = 384;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxRec = 32;                     // segments a CTA lists at a time
// A segment's beginning and end, in chunks: 1, 2, 3 and 4 are 29.9, 27.7, 27.1 and 27.3 us
// with 128 contexts at ratio 128, 75.6, 74.5, 74.2 and 73.6 with 32 long ones, 80.0, 76.7,
// 75.5 and 77.2 with 128-head drafts.
constexpr int kSegCost = 3;
// Chunks a token may exceed the mean before tokens are cut: with 6 a token of 6 chunks by
// itself takes 13.4 us instead of 9.7 (16 heads, f32 output: 14.6 and 8.9); 2, 3 and 4 are
// alike.
constexpr int kCutAbove = 4;
// Chunks between roundings of the accumulator, at most: what the tensor cores drop grows
// with the products that are added in a row (six or three terms, 64 rows).
constexpr int kFlushF32 = 27, kFlushBf16 = 341;
constexpr float kTop = 7.f;                     // log2 of the weight that the maximum is brought to

// mbar_wait whose loop is a call: the first try is nearly all that stays in line (what
// the roles run together is more than the instruction caches next to the schedulers
// hold; 32 contexts 74.2 us, with the loop in line 75.5).
__device__ __noinline__ void wait_slowly(uint64_t *bar, uint32_t parity, int32_t *status) {
    mbar_wait(bar, parity, status);
}
__device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity, int32_t *status) {
    if (__builtin_expect(!mbar_try_wait(bar, parity), 0)) wait_slowly(bar, parity, status);
}

struct PagedFp8Args : PagedArgs {
    const uint8_t *codes;
    const float *scales, *swa_scales;
    int64_t scale_stride;
    const __nv_bfloat16 *q;
};

struct Smem {
    uint64_t q_full;
    uint64_t full[kMaxStages], empty[kMaxStages][kSteps];    // a stage is released 32 rows at a time
    uint64_t sfull[2], sfree[2];
    uint64_t pfull[2][kSteps], pfree[2];
    uint32_t tmem_holder;
    uint32_t maskw[kMaxStages][kSteps];
    uint32_t risen[4];           // heads to be rescaled, 16 a word
    float alpha[kHG];            // ... and by what
    float rise[2][kHG];          // the two halves' maxima, where one rose too far
    float part_l[kHG];           // the second half's sum of weights
    float q_scale[kHG];          // a head's factor from sums of codes to logits (log2 units)
    alignas(16) float scale[kMaxStages][kChunk];   // of a row (absent rows: 0),
    alignas(16) float scale_log[kMaxStages][kChunk];   // and its logarithm;
    float log_top[kMaxStages][kSteps];                 // the largest of 32 rows, rounded up
    alignas(16) float fin[kHG];        // of a stretch: factors of the output,
    alignas(16) float flush[kHG];      // and of the partial so far
    WorkSmem<kMaxRec> work;
};


// Whether a thread of the softmax says so, behind a barrier of all of them.
__device__ __forceinline__ bool any_of(bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(mine)), "n"(kBarSm), "n"(kSmThreads)
        : "memory");
    return any != 0;
}

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

// Two f32 operations an instruction.
union Pair {
    float2 v;
    uint64_t u;
};
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    Pair x{a}, y{b}, r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(x.u), "l"(y.u));
    return r.v;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    Pair x{a}, y{b}, r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(x.u), "l"(y.u));
    return r.v;
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
__device__ __forceinline__ uint32_t f16x2_add(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// to magnitudes of at most `most`
__device__ __forceinline__ uint32_t f16x2_clamp(uint32_t a, uint32_t most) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tmin.f16x2 t, %1, %2;\n\tmax.f16x2 %0, t, %3;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(most), "r"(most | 0x80008000u));
    return r;
}
// the nearest e4m3 values of two f16, the first in the low byte
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
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
// The last term: rounded, by half of the byte's last place (an addition; the
// conversion instructions run at a quarter of its rate).  What that adds to or drops
// from a weight at e5m2's last place, 2^-16, enters the same thread's weight four rows
// on (`carry`): a sum of small weights is off by half a last place a sequence of rows,
// not one a row, which equal weights would add up: one row and 60,000 others of 2^-12 to
// 2^-22 of its weight, f32 output off by up to 2.5e-5 instead of 2.5e-3.  Above it
// the rounding is the weight's own, 2^-9 or 2^-18 of it, and kCarry bounds what is handed
// on.  32 contexts take 73.9 us instead of 73.5, 128-head drafts 75.2 instead of 74.5.  (The
// maximum brought to 2^10 and rescaled above 2^5.75, 2^13 and 2^2.75: a last place 2^-3 or
// 2^-6 of this one, 32 contexts 77.4 and 89.0 us, drafts 77.7 and 85.7.)
// (A little less than half a last place: with all of it, which a large weight's rounding
// leaves, rows without weight get 2^-16 and -2^-16 by turns; 131,008 of them beside 64
// others, f32 output off by 7.5e-6 instead of 1.1e-6.)
constexpr uint32_t kCarry = 0x007F007Fu;          // 127/128 of 2^-17, twice
__device__ __forceinline__ uint32_t last_bytes(uint32_t a, uint32_t b, uint32_t (&carry)[2]) {
    a = f16x2_add(a, carry[0]);
    b = f16x2_add(b, carry[1]);
    const uint32_t ta = (a + 0x00800080u) & 0xFF00FF00u, tb = (b + 0x00800080u) & 0xFF00FF00u;
    carry[0] = f16x2_clamp(f16x2_sub(a, ta), kCarry);
    carry[1] = f16x2_clamp(f16x2_sub(b, tb), kCarry);
    return __byte_perm(ta, tb, 0x7531);
}

// What a head's 16 sequences (four of each thread) begin with, from -120/256 to 120/256
// of a last place: equal weights are not rounded alike in all of them, and what is
// left over at their ends cancels.
__device__ __forceinline__ uint32_t first_carry(int at) {
    const int v = 8 * (2 * at - 15);
    return v < 0 ? 0x8000u | -v : v;
}

// Four weights as kTerms words of four e5m2 values each.
template <int kTerms>
__device__ __forceinline__ void split_weights(const float (&p)[4], uint32_t (&t)[kTerms], uint32_t (&carry)[2]) {
    uint32_t a = f16x2(p[0], p[1]), b = f16x2(p[2], p[3]);
    if constexpr (kTerms == 3) {
        t[0] = upper_bytes(a, b);
        t[1] = upper_bytes(a, b);
        t[2] = last_bytes(a, b, carry);
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
        t[5] = last_bytes(a, b, carry);
    }
}

// 16 columns of a head of the query as codes hi and lo.  Returns the factor that takes
// sums of codes back to the query's units (NaN where the query is not finite).  (Two
// numbers at a time by conversions; by integer operations on their bits, 12 instead of 10
// instructions, the 64 heads took 5,000 cycles instead of 4,000.)
__device__ __forceinline__ float split_query(const uint4 &v0, const uint4 &v1, uint4 &hi, uint4 &lo) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    // 1.m 2^(e - 127) to 2^7 (f16 holds what e4m3's terms need: down to 2^-14, and
    // 8 bits), as far as a factor of 2^126 does it: below 2^-119 a head keeps fewer bits
    const int k = min(134 - static_cast<int>(top >> 7), 126);
    const float f = exponent_f32(k);
    const float2 s1 = make_float2(f, f);
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 x = mul2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), s1);
        const uint32_t y = f16x2(x.x, x.y);
        h[i] = f16x2_e4m3x2(y);
        l[i] = f16x2_e4m3x2(f16x2_sub(y, e4m3x2_f16x2(h[i])));
    }
    hi = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    lo = make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
    return top >= 0x7F80u ? NAN : exponent_f32(-k);
}

// A load under a condition that nothing waits for until the result is used (where a
// branch's two ends are joined by a move, that does).
template <bool kL2>
__device__ __forceinline__ int32_t load_if(const void *p, bool ok) {
    int32_t r;
    if constexpr (kL2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.cg.b32 %0, [%1];\n\t}"
                     : "=r"(r) : "l"(p), "r"(static_cast<uint32_t>(ok)));
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.b32 %0, [%1];\n\t}"
                     : "=r"(r) : "l"(p), "r"(static_cast<uint32_t>(ok)));
    return r;
}

// A contiguous copy into shared memory, a multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// The barrier's phase waits for this thread's cp.async copies too.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// One 32-bit column of tensor memory, a lane a thread.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(x)) : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns from registers
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// kTerms: e5m2 terms of P (6 for an f32 output, 3 for bf16).
template <int kTerms>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_fp8_kernel(const __grid_constant__ CUtensorMap tm_rows, const PagedFp8Args A) {
    constexpr bool kBf16 = kTerms == 3;
    constexpr int kFlush = kBf16 ? kFlushBf16 : kFlushF32;
    constexpr int kPiece = kPieceBytes<kTerms>;          // 16 rows of P
    constexpr int kSt = kStages<kTerms>, kPB = kPBufs, kSB = kSBufs<kTerms>;
    constexpr int kWd = kWide<kTerms>, kO = kOCol<kTerms>;
    auto o_col = [](int dd) { return kO + kHG * (dd + (dd < kWd ? dd : kWd)); };
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align_smem<1024>(smem_raw);
    uint8_t *sRows = smem;                               // [stage][8 groups][4 col groups][8 rows][128 B]
    uint8_t *sP = sRows + kSt * kStageBytes;             // [buffer][16 rows of the chunk][term][64 heads][16 B]
    Smem &S = *reinterpret_cast<Smem *>(sP + kPB * (kChunk / 16) * kPiece);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hg = blockIdx.y, h0 = hg * kHG;
    const int H = A.H;

    if (tid == 0) {
        mbar_init(&S.q_full, kSmThreads);
        for (int i = 0; i < kSt; ++i) {
            mbar_init(&S.full[i], kSteps);
            for (int k = 0; k < kSteps; ++k) mbar_init(&S.empty[i][k], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.sfree[i], kSmThreads);
            for (int k = 0; k < kSteps; ++k) mbar_init(&S.pfull[i][k], kSmGroup);
            mbar_init(&S.pfree[i], 1);
        }
        mbar_fence_init();
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
    const int ndt = W.ndt, dt0 = W.dt0;                  // 128-column tiles of this CTA
    const Rec *const rec = S.work.rec;

    // pipeline positions, kept across lists of segments
    uint32_t n_fetch = 0;                // chunks fetched
    uint32_t nq = 0, np = 0;             // chunks whose S / O^T products were issued
    // (a segment's query passes through two stages, ahead of its chunks, so that
    // chunk n of segment m is number n + 2 m + 2 of what the stages hold)
    uint32_t n_ql = 0;                   // segments begun
    uint32_t n_sm = 0;                   // chunks through the softmax

    for (;;) {
        __syncthreads();
        W.advance();
        const int nrec = S.work.nrec;
        const bool more = S.work.more != 0;
        if (nrec == 0) break;

        if (warp == 8) {
            // -------------------------------------------- S = Q . rows^T
            // A whole warp keeps step and one elected thread issues, here and below.
            constexpr uint32_t id = idesc_fp8<2 * kHG, kChunk, false, false>();
            const uint64_t r_desc = sw128_desc(smem_addr(sRows), 16, kGroupBytes);
            for (int i = 0; i < nrec; ++i) {
                const int nch = rec[i].c1 - rec[i].c0;
                if (nch <= 0) continue;
                wait_for(&S.q_full, n_ql & 1u, A.status);
                ++n_ql;
                for (int k = 0; k < nch; ++k, ++nq) {
                    const uint32_t slot = nq + 2 * n_ql;
                    const uint32_t st = slot % kSt, sb = nq % kSB;
                    wait_for(&S.full[st], (slot / kSt) & 1u, A.status);
                    wait_for(&S.sfree[sb], ((nq / kSB) & 1u) ^ 1u, A.status);
                    fence_proxy_async_smem();            // (rows that came one by one)
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
                        uint64_t rd = r_desc + off(st * kStageBytes);
                        uint32_t qa = tmem + kQCol;
                        const uint32_t d = tmem + kSCol + sb * 64;
#pragma unroll 1
                        for (int cg = 0; cg < kHD / 128; ++cg, qa += 32, rd += off(1024)) {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                umma_fp8_ts(d, qa + 8 * x, rd + off(x * 32), id, x > 0 ? 1u : cg);
                        }
                        umma_commit(&S.sfull[sb]);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 9) {
            // -------------------------------------------- O^T += rows^T . P^T
            constexpr uint32_t id = idesc_fp8<128, kHG, true, true>(), id_wide = idesc_fp8<128, 2 * kHG, true, true>();
            const uint64_t a_desc = sw128_desc(smem_addr(sRows) + dt0 * 1024, 1024, kGroupBytes);
            const uint64_t p_desc = atom_desc(smem_addr(sP), kPiece, 128);
            auto product = [&](int dd, uint64_t ad, uint64_t pd, uint32_t acc) {
                if (dd < kWd) {
#pragma unroll
                    for (int t = 0; t < kTerms; t += 2)
                        umma_fp8(tmem + o_col(dd), ad + off(dd * 1024), pd + off(t * kTermBytes), t + 1 < kTerms ? id_wide : id,
                                 t > 0 ? 1u : acc);
                } else {
#pragma unroll
                    for (int t = 0; t < kTerms; ++t)
                        umma_fp8(tmem + o_col(dd), ad + off(dd * 1024), pd + off(t * kTermBytes), id, t > 0 ? 1u : acc);
                }
            };
            for (int i = 0; i < nrec; ++i) {
                const int nch = rec[i].c1 - rec[i].c0;
                if (nch <= 0) continue;
                ++n_ql;
                const int every = flush_every<kFlush>(nch);
                for (int k = 0, z = 0; k < nch; ++k, ++np, z = z + 1 == every ? 0 : z + 1) {
                    const uint32_t st = (np + 2 * n_ql) % kSt, pb = np % kPB;
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        const uint64_t ad = a_desc + off(st * kStageBytes + ks * 4 * kGroupBytes);
                        const uint64_t pd = p_desc + off((pb * (kChunk / 16) + 2 * ks) * kPiece);
                        wait_for(&S.pfull[pb][ks], (np / kPB) & 1u, A.status);
                        // (a stretch's first product: the one before it has been drained by the
                        // warps that made these weights)
                        const uint32_t acc = z > 0 || ks > 0;
                        __syncwarp();
                        tc_fence_after();
                        if (elect_one()) {
                            // (all columns, unrolled: the loop's issue alone holds the tensor
                            // cores up, 32 contexts 74.9 us instead of 74.2, drafts 76.7 and 75.5)
                            if (ndt == 4) {
#pragma unroll
                                for (int dd = 0; dd < 4; ++dd) product(dd, ad, pd, acc);
                            } else {
#pragma unroll 1
                                for (int dd = 0; dd < ndt; ++dd) product(dd, ad, pd, acc);
                            }
                        }
                        __syncwarp();
                        if (elect_one()) {
                            umma_commit(&S.empty[st][ks]);
                            if (ks + 1 == kSteps) umma_commit(&S.pfree[pb]);
                        }
                        __syncwarp();
                    }
                }
            }
        } else if (warp >= 10) {
            // -------------------------------------------- row fetch
            // The warp walks the list's chunks, a row of each a lane: two chunks before it
            // is copied its page number is on its way from the table, one before it its
            // scale.  (Whole chunks by turns, two rows a lane, took as long in the loop, but a
            // call's first rows started later: 256 rows 10.7 us instead of 9.6.)
            const int li = warp - 10;
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
                int32_t page, at;                      // the table's entry; row of the page or of the rings, < 0: no row
                bool ring, box;                        // 8 rows of one page from here on
            };
            auto look_up = [&](const Cursor &k) {
                Entry e{-1, -1, false, false};
                if (k.i >= nrec) return e;
                const Rec &r = rec[k.i];
                const int j = k.c * kChunk + 32 * li + lane, w = j - rec_window_slot(r);
                const bool in = j < r.n;
                const int pg = static_cast<int>(A.page_div.div(in ? j : 0));
                e.page = load_if<false>(A.L.table + static_cast<int64_t>(r.b) * A.L.max_pages + pg, in);
                const int at = j - pg * A.L.page_rows;
                if (in) e.at = at;
                e.box = in && j + 8 <= r.n && at + 8 <= A.L.page_rows;
                if (!in && w >= 0 && w < r.near) {
                    const int64_t x = r.first + w;
                    e.ring = true;
                    if (x < r.first_res) bad |= CSA_DEV_MISSING_SWA;
                    else e.at = r.b * A.L.swa_cap + static_cast<int32_t>(A.swa_div.mod64(x));
                }
                return e;
            };
            struct Place {
                int32_t row;                           // of the pool or of the rings, or -1
                float scale;
                uint32_t box;                          // bit 8 g: group g of 8 rows is one box
                uint32_t ring;                         // ... of the rings (no group holds rows of both)
            };
            auto place = [&](const Entry &e) {
                Place p;
                const bool paged = e.at >= 0 && !e.ring;
                const bool out = paged && static_cast<uint32_t>(e.page) >= static_cast<uint32_t>(A.num_pages);
                p.row = e.ring ? e.at : static_cast<int32_t>(e.page * A.page_stride) + e.at;
                if (out) bad |= CSA_DEV_BAD_INDEX;
                if (e.at < 0 || out) p.row = -1;
                if (!CSA_CHECK(e.ring || p.row < A.total_rows, A.status)) p.row = -1;
                p.scale = __int_as_float(load_if<true>(
                    e.ring ? A.swa_scales + e.at : A.scales + e.page * A.scale_stride + e.at, p.row >= 0));
                p.box = __ballot_sync(0xffffffffu, e.box) & 0x01010101u;
                p.ring = __ballot_sync(0xffffffffu, e.ring);
                return p;
            };
            // rows are read once, or once by each of two groups of heads
            const uint64_t pol = gridDim.y > 1 ? policy_evict_normal() : policy_evict_first();
            Cursor cur{0, rec[0].c0};
            settle(cur);
            Cursor far = cur;
            // the query of a segment: two stages ahead of its rows, 32 heads each
            int of = -1;                               // the segment whose query has been fetched
            auto query = [&](int i) {
                of = i;
#pragma unroll 1
                for (int x = 0; x < 2; ++x, ++n_fetch) {
                    // (the whole stage, which the other warp's rows may still be in)
                    for (int k = 0; k < kSteps; ++k)
                        wait_for(&S.empty[n_fetch % kSt][k], ((n_fetch / kSt) & 1u) ^ 1u, A.status);
                    __syncwarp();
                    if (lane == 0) {
                        uint64_t *const full = &S.full[n_fetch % kSt];
                        const int h = h0 + 32 * x, heads = min(32, H - h);
                        if (li == 0 && heads > 0) {
                            mbar_expect_tx(full, heads * kHD * 2);
                            bulk_load(sRows + n_fetch % kSt * kStageBytes,
                                      A.q + (static_cast<int64_t>(rec[i].t) * H + h) * kHD, heads * kHD * 2, full);
                        }
                        mbar_arrive(full);
                    }
                }
            };
            if (cur.i < nrec) query(cur.i);
            Place now{}, next{};
            Entry ahead{-1, -1, false, false};
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                now = next;
                next = place(ahead);
                ahead = look_up(far);
                advance(far);
            }
            while (cur.i < nrec) {
                // (the queue moves up first: the loads that it starts take as long as the
                // stage's wait)
                now = next;
                next = place(ahead);
                ahead = look_up(far);
                advance(far);
                if (cur.i != of) query(cur.i);
                const uint32_t okm = __ballot_sync(0xffffffffu, now.row >= 0);
                const int32_t y = __shfl_sync(0xffffffffu, now.row, (8 * lane) & 31);     // of group `lane`
                const int st = n_fetch % kSt;
                const uint32_t ph = ((n_fetch / kSt) & 1u) ^ 1u;
                uint64_t *const empty = &S.empty[st][li], *const full = &S.full[st];
                wait_for(empty, ph, A.status);
                __syncwarp();
                uint8_t *rows = sRows + st * kStageBytes + 4 * li * kGroupBytes;
                if (lane == 0) {
                    S.maskw[st][li] = okm;
                    if (now.box) mbar_expect_tx(full, __popc(now.box) * kGroupBytes);
                }
                __syncwarp();
                // (a bad page: a box behind the pool reads as zeros)
                if (lane < 4 && (now.box >> (8 * lane) & 1u))
                    tma_load_3d(rows + lane * kGroupBytes, &tm_rows, 0, y >= 0 ? y : A.total_rows, 0, full, pol);
                if (now.box != 0x01010101u) {
                    // eight lanes take 128 columns of a row, four rows an instruction (a row an
                    // instruction, 128 contexts in pages of two rows, were 28.6 us instead of 27.7)
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        if (now.box >> (8 * x) & 1u) continue;
                        const uint8_t *const from =
                            (now.ring >> (8 * x) & 1u ? static_cast<const uint8_t *>(A.L.swa_kv) : A.codes) + (lane & 7) * 16;
                        uint8_t *const to = rows + x * kGroupBytes;
#pragma unroll
                        for (int h = 0; h < 8; h += 4) {
                            const int rr = h + (lane >> 3);
                            const int32_t row = __shfl_sync(0xffffffffu, now.row, 8 * x + rr);
                            const uint8_t *const src = from + static_cast<int64_t>(max(row, 0)) * kHD;
                            uint8_t *const dst = to + rr * 128 + (((lane & 7) ^ rr) << 4);
#pragma unroll
                            for (int cg = 0; cg < 4; ++cg) cp_async16(dst + cg * 1024, src + cg * 128, row >= 0);
                        }
                    }
                    // (the stage is full when they have landed; nobody waits for them here)
                    cp_async_arrive(full);
                }
                // (behind the copies: a scale may still be on its way)
                const float slog = now.row >= 0 ? __log2f(fminf(fmaxf(fabsf(now.scale), 0x1p-60f), 0x1p60f)) : 0.f;
                // (in whole powers of two; the hundredth takes a power's own error)
                const float log_top = static_cast<int>(__reduce_max_sync(
                    0xffffffffu, now.row >= 0 ? static_cast<unsigned>(__float2int_ru(slog - 0.01f) + 64) : 0u)) - 64;
                S.scale[st][32 * li + lane] = now.scale;
                S.scale_log[st][32 * li + lane] = slog;
                if (lane == 0) S.log_top[st][li] = log_top;
                advance(cur);
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
                ++n_fetch;
            }
            bad = static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad)));
            if (lane == 0 && W.lead) raise_status(A.status, bad);
        } else {
            // -------------------------------------------- the query, softmax
            const int q = warp & 3;                  // TMEM lane quarter
            const int g = warp >> 2;                 // rows 0..31 of a chunk, or 32..63
            const int hl = q * 16 + (lane & 15);     // head of this lane (four lanes per head, two of each half)
            const bool upper = lane >= 16;           // the second 16 of those rows
            const int r0 = 32 * g + (upper ? 16 : 0);
            const bool hv = h0 + hl < H;
            const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
            // O^T of the stretch whose last chunk was the one before n_sm, into the partial
            // or the output; each half of the warps takes 32 heads
            auto drain = [&](int of, bool add, bool part) {
                const Rec &r = rec[of];
                (void)CSA_CHECK(r.slot < 2 * W.G && r.t < W.T, A.status);
                wait_for(&S.pfree[(n_sm - 1) % kPB], ((n_sm - 1) / kPB) & 1u, A.status);
                __syncwarp();
                named_bar_sync(kBarSm, kSmThreads);      // (the factors are written)
                tc_fence_after();
                drain_stretch<kBf16, kWd, kStagedHeads>(
                    A, tmem + lane_off + kO, S.fin, S.flush, nullptr, sP + warp * staged_bytes(kStagedHeads), dt0, ndt,
                    32 * g, 32 * g + 32, min(kHG, H - h0), (static_cast<int64_t>(r.t) * H + h0) * kHD,
                    static_cast<int64_t>(r.slot) * gridDim.y + hg, add, part);
                __syncwarp();
            };
            int left = -1;                           // the segment whose O^T is still to be drained
            bool left_add = false;
            for (int i = 0; i < nrec; ++i) {
                const int nch = rec[i].c1 - rec[i].c0;
                if (nch <= 0) {
                    if (rec[i].flags & kRecZero) {
                        const int64_t obase = (static_cast<int64_t>(rec[i].t) * H + h0) * kHD;
                        for (int x = tid; x < min(kHG, H - h0) * 128 * ndt; x += kSmThreads) {
                            const int64_t at = obase + (x / (128 * ndt)) * kHD + dt0 * 128 + x % (128 * ndt);
                            if (kBf16) static_cast<__nv_bfloat16 *>(A.out)[at] = __float2bfloat16(0.f);
                            else static_cast<float *>(A.out)[at] = 0.f;
                        }
                    }
                    continue;
                }
                // (the segment before this one is done with Q when its last logits have
                // come)
                if (n_sm > 0) wait_for(&S.sfull[(n_sm - 1) % kSB], ((n_sm - 1) / kSB) & 1u, A.status);
                __syncwarp();
                tc_fence_after();
                // The heads that there are, by turns among the warps, each split in its place
                // (a lane has 2 x 8 columns; a head's 512 codes hi, then lo, in pieces of 16
                // whose order depends on the head); then half a row of codes a lane into
                // tensor memory.  (Rows of absent heads hold anything: no other row's sums
                // see them, and their own are left where they are.)
                {
                    const uint32_t slot = n_sm + 2 * n_ql;
                    const int st0 = slot % kSt, st1 = (slot + 1) % kSt;
                    wait_for(&S.full[st0], (slot / kSt) & 1u, A.status);
                    wait_for(&S.full[st1], ((slot + 1) / kSt) & 1u, A.status);
                    __syncwarp();
                    const int heads = min(kHG, H - h0);
#pragma unroll 2
                    for (int h = warp; h < heads; h += kSmThreads / 32) {
                        uint8_t *const at = sRows + (h < 32 ? st0 : st1) * kStageBytes + (h & 31) * 1024;
                        const uint4 v0 = reinterpret_cast<const uint4 *>(at)[lane];
                        const uint4 v1 = reinterpret_cast<const uint4 *>(at)[32 + lane];
                        uint4 hi, lo;
                        const float f = split_query(v0, v1, hi, lo);
                        __syncwarp();
                        uint2 *const to = reinterpret_cast<uint2 *>(at) + (lane ^ (h & 7) << 1);
                        to[0] = make_uint2(hi.x, hi.y);
                        to[32] = make_uint2(hi.z, hi.w);
                        to[64] = make_uint2(lo.x, lo.y);
                        to[96] = make_uint2(lo.z, lo.w);
                        if (lane == 0) S.q_scale[h] = f * A.scale_log2;
                    }
                    __syncwarp();
                    named_bar_sync(kBarSm, kSmThreads);
                    const uint4 *const get = reinterpret_cast<const uint4 *>(
                        sRows + (q < 2 ? st0 : st1) * kStageBytes + ((q & 1) * 16 + (lane & 15)) * 1024 + (lane >> 4) * 512) + 16 * g;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        if (16 * q >= heads) break;
                        uint32_t o[32];
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const uint4 u = get[(8 * half + x) ^ (lane & 7)];
                            o[4 * x] = u.x;
                            o[4 * x + 1] = u.y;
                            o[4 * x + 2] = u.z;
                            o[4 * x + 3] = u.w;
                        }
                        tmem_st32(tmem + lane_off + kQCol + 64 * g + 32 * half, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    fence_proxy_async_smem();
                    mbar_arrive(&S.q_full);
                    wait_for(&S.q_full, n_ql & 1u, A.status);       // (all are done: the stages go back)
                    if (tid == 0)
                        for (int k = 0; k < kSteps; ++k) {
                            mbar_arrive(&S.empty[st0][k]);
                            mbar_arrive(&S.empty[st1][k]);
                        }
                    __syncwarp();
                }
                ++n_ql;
                // the segment before this one, under this one's first logits
                if (left >= 0) drain(left, left_add, rec[left].flags & kRecPart);
                const float c = S.q_scale[hl];

                const bool cut = rec[i].flags & kRecPart;
                float m_ref = -INFINITY, l = 0.f, l_all = 0.f, m_flush = -INFINITY;
                const int sq = 4 * (2 * g + (upper ? 1 : 0));
                // (kept where a maximum rises: at most half a last place)
                uint32_t carry[2] = {first_carry(sq) | first_carry(sq + 1) << 16,
                                     first_carry(sq + 2) | first_carry(sq + 3) << 16};
                const int every = flush_every<kFlush>(nch);
                const float2 c2 = make_float2(c, c);
                for (int k = 0, z = 0; k < nch; ++k, ++n_sm, z = z + 1 == every ? 0 : z + 1) {
                    const uint32_t slot = n_sm + 2 * n_ql;
                    const int st = slot % kSt, sb = n_sm % kSB;
                    // the rows' masks and scales, before their logits come
                    wait_for(&S.full[st], (slot / kSt) & 1u, A.status);
                    const uint32_t mw = S.maskw[st][g] >> (r0 & 16) & 0xFFFFu;
                    const float log_top = S.log_top[st][g];
                    float2 s[8], x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float4 *>(s + 2 * j) = *reinterpret_cast<const float4 *>(S.scale[st] + r0 + 4 * j);
                    // (a wait's lanes may leave it at different polls; what is
                    // .aligned below, tensor memory and barriers, wants the warp whole)
                    wait_for(&S.sfull[sb], (n_sm / kSB) & 1u, A.status);
                    __syncwarp();
                    tc_fence_after();
                    {
                        uint32_t hi[16], lo[16];
                        const uint32_t at = tmem + lane_off + kSCol + sb * 64 + 32 * g;
                        tmem_ld16x2_next_raw(at, hi);
                        tmem_ld16x2_next_raw(at + (16u << 16), lo);
                        tmem_wait_ld();
                        tc_fence_before();
                        mbar_arrive(&S.sfree[sb]);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = mul2(add2(make_float2(__uint_as_float(hi[2 * j]), __uint_as_float(hi[2 * j + 1])),
                                             make_float2(__uint_as_float(lo[2 * j]), __uint_as_float(lo[2 * j + 1]))),
                                        mul2(s[j], c2));
                    }
                    if (__any_sync(0xffffffffu, mw != 0xFFFFu)) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (!(mw >> (2 * j) & 1u)) x[j].x = -INFINITY;
                            if (!(mw >> (2 * j + 1) & 1u)) x[j].y = -INFINITY;
                        }
                    }
                    // The maximum is that of the logits plus their scales' logarithms; a head whose
                    // maximum rises by more than kRescaleAbove (the first one does) rescales
                    // what has been accumulated.  The largest logit plus the largest logarithm
                    // of the 32 rows tells nearly always that none does.  (With every row's
                    // logarithm read in every chunk one million tokens take 44.9 us instead of
                    // 43.6, 32 contexts 77.2 instead of 74.2, but 8,192 rows 14.1 instead of 14.2.)
                    float mc = fmaxf(x[0].x, x[0].y);
#pragma unroll
                    for (int j = 1; j < 8; ++j) mc = fmaxf(mc, fmaxf(x[j].x, x[j].y));
                    bool risen = false;
                    float alpha = 1.f;
                    if (k == 0 || any_of(hv && mc + log_top > m_ref + kRescaleAbove)) {
                        mc = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 y = *reinterpret_cast<const float4 *>(S.scale_log[st] + r0 + 4 * j);
                            mc = fmaxf(fmaxf(mc, fmaxf(x[2 * j].x + y.x, x[2 * j].y + y.y)),
                                       fmaxf(x[2 * j + 1].x + y.z, x[2 * j + 1].y + y.w));
                        }
                        mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, 16));
                        risen = k == 0 || any_of(hv && mc > m_ref + kRescaleAbove);
                    }
                    if (risen) {
                        if (!upper) S.rise[g][hl] = mc;
                        __syncwarp();
                        named_bar_sync(kBarSm, kSmThreads);
                        mc = fmaxf(S.rise[0][hl], S.rise[1][hl]);
                        if (hv && mc > m_ref + kRescaleAbove) {
                            if (m_ref != -INFINITY) alpha = exp2f(m_ref - mc);
                            m_ref = mc;
                            l *= alpha;
                            l_all *= alpha;
                        }
                    }
                    const float mr = m_ref == -INFINITY ? 0.f : m_ref - kTop;
                    const float2 m2 = make_float2(-mr, -mr);
                    float2 sum = make_float2(0.f, 0.f);
                    uint32_t w[4][kTerms];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float2 v = add2(x[2 * u + e], m2);
                            v = make_float2(fast_exp2(v.x), fast_exp2(v.y));
                            sum = add2(sum, v);
                            v = mul2(v, s[2 * u + e]);
                            p[2 * e] = v.x;
                            p[2 * e + 1] = v.y;
                        }
                        split_weights<kTerms>(p, w[u], carry);
                    }
                    l += sum.x + sum.y;
                    const int pb = n_sm % kPB;
                    wait_for(&S.pfree[pb], ((n_sm / kPB) & 1u) ^ 1u, A.status);
                    uint8_t *const at = sP + (pb * (kChunk / 16) + 2 * g + (upper ? 1 : 0)) * kPiece + hl * 16;
#pragma unroll
                    for (int t = 0; t < kTerms; ++t)
                        *reinterpret_cast<uint4 *>(at + t * kTermBytes) = make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]);
                    if (risen && z != 0) {
                        const uint32_t mine = __ballot_sync(0xffffffffu, alpha != 1.f) & 0xFFFFu;
                        if (g == 0 && !upper) S.alpha[hl] = alpha;
                        if (g == 0 && lane == 0) S.risen[q] = mine;
                        // (the weights are made meanwhile; the product before this one)
                        wait_for(&S.pfree[(n_sm - 1) % kPB], ((n_sm - 1) / kPB) & 1u, A.status);
                        __syncwarp();
                        named_bar_sync(kBarSm, kSmThreads);
                        tc_fence_after();
                        // head by head (seldom more than a few), a tile or two a half of
                        // the warps
                        uint64_t heads = S.risen[0] | static_cast<uint64_t>(S.risen[1]) << 16 |
                                         static_cast<uint64_t>(S.risen[2]) << 32 | static_cast<uint64_t>(S.risen[3]) << 48;
                        while (heads) {
                            const int h = __ffsll(heads) - 1;
                            heads &= heads - 1;
                            const uint32_t o = tmem + lane_off + h;
                            const float f = S.alpha[h];
                            const int dd = ndt == 4 ? 2 * g : g;
                            const uint32_t a = o + o_col(dd), b = o + o_col(dd + 1);
                            if (dd < kWd) {                    // (its second half)
                                const float x = tmem_ld1(a + kHG);
                                tmem_wait_ld();
                                tmem_st1(a + kHG, x * f);
                            }
                            if (ndt == 4) {
                                const float x0 = tmem_ld1(a), x1 = tmem_ld1(b);
                                tmem_wait_ld();
                                tmem_st1(a, x0 * f);
                                tmem_st1(b, x1 * f);
                            } else if (dd < ndt) {
                                const float x0 = tmem_ld1(a);
                                tmem_wait_ld();
                                tmem_st1(a, x0 * f);
                            }
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        named_bar_sync(kBarSm, kSmThreads);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&S.pfull[pb][g]);

                    const bool last = k + 1 == nch;
                    if (!last && z + 1 != every) continue;
                    // the weights' sum, as their products with the rows: every stretch is a
                    // sum of its own (equal weights beside a large one are rounded alike:
                    // added chunk by chunk, 262,144 rows left an f32 output off by 1.5e-4
                    // instead of 4.3e-5)
                    l_all += l;
                    l = 0.f;
                    if (last) {
                        l = l_all;
                        __syncwarp();
                        l += __shfl_xor_sync(0xffffffffu, l, 16);
                        if (g == 1 && !upper) S.part_l[hl] = l;
                        named_bar_sync(kBarSm, kSmThreads);
                        if (g == 0) l += S.part_l[hl];
                    }
                    // the stretch's factors for the epilogue
                    if (g == 0 && !upper) {
                        S.flush[hl] = m_flush == -INFINITY ? 1.f : exp2f(m_flush - m_ref);
                        float f = 1.f;
                        if (last && !cut) {
                            float zs = l;
                            if (A.sinks && hv) zs += exp2f(A.sinks[h0 + hl] * kLog2e - mr);
                            f = m_ref == -INFINITY && l == 0.f ? 0.f : 1.f / zs;     // (a sink of NaN: NaN)
                        }
                        S.fin[hl] = f;
                        if (last && cut && dt0 == 0)
                            A.part_ml[(static_cast<int64_t>(rec[i].slot) * gridDim.y + hg) * kHG + hl] =
                                make_float2(m_ref == -INFINITY ? m_ref : mr, l);
                    }
                    m_flush = m_ref;
                    __syncwarp();
                    if (last) {
                        left = i;
                        left_add = k >= every;           // the partial holds earlier stretches
                    } else {
                        ++n_sm;
                        drain(i, k >= every, true);
                        --n_sm;
                    }
                }
            }
            if (left >= 0) drain(left, left_add, rec[left].flags & kRecPart);
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
constexpr size_t smem_bytes() {
    return 1024 + kStages<kTerms> * kStageBytes + kPBufs * (kChunk / 16) * kPieceBytes<kTerms> + sizeof(Smem);
}
static_assert(smem_bytes<3>() <= 227 * 1024 && smem_bytes<6>() <= 227 * 1024);

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
