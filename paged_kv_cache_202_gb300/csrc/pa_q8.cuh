// Conversions and the row mapping shared by the kernels of the 8-bit cache.
#pragma once

#include <cfloat>
#include <cstdint>

#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace q8 {

// Two e4m3 codes (the low one in the low byte) as two halves: exact, NaN to NaN.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t codes16) {
    uint32_t r;
    asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {c, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes16));
    return r;
}

__device__ __forceinline__ uint32_t hi_to_f16x2(uint32_t codes32) {
    uint32_t r;
    asm("{\n\t.reg .b16 c, u;\n\tmov.b32 {u, c}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes32));
    return r;
}

// Two floats as two codes, nearest even, saturating at 448 (NaN to NaN).
__device__ __forceinline__ uint32_t from_f32x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t from_f32x4(float a, float b, float c, float d) {
    return from_f32x2(a, b) | from_f32x2(c, d) << 16;
}

// Two halves as two floats.
__device__ __forceinline__ float2 f16x2_split(uint32_t h) {
    float2 v;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}

// The smallest power of two s with a <= 448 s, at least 2^-64 (2^(least - 127); a >= 0, finite):
// 448 = 1.75 x 2^8, so s is 2^(e - 8) for a = m 2^e with m <= 1.75, else 2^(e - 7).
__device__ __forceinline__ float scale_for(float a, uint32_t least = 63u) {
    const uint32_t e = (__float_as_uint(a) + 0x1fffffu) >> 23;  // one more above mantissa 1.75
    return __uint_as_float((e < least + 8u ? least : e - 8u) << 23);
}

// The value scales that the attention takes: those that pa_qk_rope_append_q8 makes. Weights
// carry the value scale of their token, w = 2^(s + log2 vs - m), and their sum does not,
// l = sum of w / vs = sum of 2^(s - m), which spans 2^184 against the largest w. So l is
// taken times 2^24, between 2^-89 and 2^103 a token. While the scales of a segment lie
// within 2^90 of one another, a token whose w is below float's range is worth less than
// 2^-43 of l. From the first page on that lies further apart (`far`), l takes 2^(s - m)
// itself, and is brought to another m in two steps.
constexpr float kMinValueScale = 0x1p-64f, kMaxValueScale = 0x1p120f;
constexpr float kFarApart = 90.f, kSumBias = 24.f, kSumFactor = 0x1p24f;

// log2 of a block's value scale; NaN, which shows in the rows, for scales that are none.
__device__ __forceinline__ float log2_of(float vs, float ks) {
    const bool fine = vs >= kMinValueScale && vs <= kMaxValueScale && ks > 0.f && ks <= FLT_MAX;
    return fine ? fast_log2(vs) : __int_as_float(0x7fc00000);
}

// f 2^d for a 2^d that may be below float's range while the product is not.
__device__ __forceinline__ float times_exp2(float f, float d) {
    const float h = fast_exp2(0.5f * d);
    return f * h * h;
}

// The work of a call on the blocks that hold its rows. Sequence b's rows lie in at
// most rows / block_size + 2 blocks, so item x = (q_start[b] >> shift) + 2 b + j is
// its j-th block, whatever the other sequences have: no list of items has to be
// built, and (num_rows >> shift) + 2 B items hold them all. Items past a
// sequence's last block are empty.
struct Rows {
    int b, phys;       // sequence; block in the pools
    int row0, n;       // its rows of the call: row0 .. row0 + n - 1
    int off0;          // offset of the first in the block
};

struct RowArgs {
    const int32_t* q_start;   // [B + 1]
    const int32_t* tables;
    const int32_t* seq_lens;
    int* err;
    int B, T, max_blocks, num_blocks, shift;
};

// Whether sequence b's rows and length are in range (n_b may be 0).
__device__ __forceinline__ bool rows_ok(const RowArgs& a, int q0, int q1, int L) {
    return q0 >= 0 && q1 >= q0 && q1 <= a.T && L >= q1 - q0 && L <= a.max_blocks << a.shift;
}

// Item x, the same in every thread of a block; false: nothing to do. `report`
// (one block of the call): raise what is wrong with any sequence's rows.
__device__ __forceinline__ bool find_rows(const RowArgs& a, int x, bool report, Rows* r) {
    if (report) {
        for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
            const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
            if (!rows_ok(a, q0, q1, a.seq_lens[b])) atomicOr(a.err, kErrSeqLen);
        }
    }
    // The last sequence whose first item is at most x. First 32 candidates around the
    // place it has when all have as many rows, with what the item needs of each; where it
    // is not among them, 32 candidates a round over all.
    const int lane = threadIdx.x & 31;
    const float share = static_cast<float>(x) * a.B / (static_cast<float>(a.T >> a.shift) + 2.f * a.B);
    const int i0 = max(0, min(static_cast<int>(share) - 16, a.B - 32)), i = min(i0 + lane, a.B - 1);
    int q0 = a.q_start[i], q1 = a.q_start[i + 1], L = a.seq_lens[i];
    uint32_t at = __ballot_sync(0xffffffffu, i0 + lane < a.B && (q0 >> a.shift) + 2 * i <= x);
    int lo = i0 + max(__popc(at), 1) - 1;
    if ((at & 1u || i0 == 0) && (!(at >> 31) || i0 + 32 >= a.B)) {
        q0 = __shfl_sync(0xffffffffu, q0, lo - i0);
        q1 = __shfl_sync(0xffffffffu, q1, lo - i0);
        L = __shfl_sync(0xffffffffu, L, lo - i0);
    } else {
        int len = a.B;
        lo = 0;
        while (len > 1) {
            const int step = (len + 31) >> 5, e = lo + lane * step;
            const bool in = lane * step < len && (a.q_start[e] >> a.shift) + 2 * e <= x;
            const int c = max(__popc(__ballot_sync(0xffffffffu, in)), 1) - 1;
            lo += c * step;
            len = min(step, len - c * step);
        }
        q0 = a.q_start[lo], q1 = a.q_start[lo + 1], L = a.seq_lens[lo];
    }
    const int j = x - (q0 >> a.shift) - 2 * lo;
    if (j < 0 || q1 == q0 || !rows_ok(a, q0, q1, L)) return false;
    const int p0 = L - (q1 - q0);
    const int blk = (p0 >> a.shift) + j;
    if (blk > (L - 1) >> a.shift) return false;
    const int first = max(p0, blk << a.shift), last = min(L, (blk + 1) << a.shift);
    r->b = lo;
    r->row0 = q0 + first - p0;
    r->n = last - first;
    r->off0 = first & ((1 << a.shift) - 1);
    r->phys = a.tables[static_cast<size_t>(lo) * a.max_blocks + blk];
    if (r->phys < 0 || r->phys >= a.num_blocks) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrTable);
        return false;
    }
    return true;
}

}  // namespace q8
}  // namespace pa
