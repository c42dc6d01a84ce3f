// Causal attention of many queries over a paged cache held in 8 bits
// (pa_prefill_q8), on the tcgen05 tensor cores.
//
// A query tile holds 128 rows = (128 / g) queries x the g query heads of a kv head
// and takes the keys and values in 128-token chunks through the block table. With kc,
// vc the codes and ks, vs the scales of a token's block,
//   s' = scale log2(e) ks (q . kc) + log2(vs),   w = 2^(s' - m),
//   O = sum w vc,   l = sum w / vs,   out = O / l
// (pa_split_q8.cu says why the values' scales sit in the exponents).
//
// Scores. The keys' codes go into the products as they are: kind::f8f6f4, e4m3 times
// e4m3. A query row, brought to at most 448 by a power of two, is the sum of two
// e4m3 numbers, hi = the nearest and lo = the nearest to the rest: bf16's 8 bits are
// 4 + 4, so that only what lies below 2^-17 of the row's largest element is rounded.
// S = Qhi K^T + Qlo K^T is one product with K = 256 at twice bf16's rate: the time of
// a bf16 product, and the keys take no instruction and half the shared memory.
// Values. Weights need more than 4 bits, so O = W V is a product of kind::f16, and
// four warps turn the codes of a chunk into f16 in shared memory (exact) while the
// tensor core works on the chunk before. W is rounded to f16, times 2^7: 11 bits, down
// to 2^-32 of the largest; l takes the weights unrounded.
//
// Measured (device time; a large bf16 product runs at 1945 TFLOP/s, 1733 sustained).
// 16384 rows of one prompt, 32 / 8 heads: 1527 to 1550 us, 1430 TFLOP/s (0.73, 0.82 of the
// sustained rate). 16 sequences of 256 rows, 1024 to 16384 tokens: 261 us, 1232 TFLOP/s.
// Bound by a tile's chain: scores, softmax, weights, value product, about 3100 cycles for
// a chunk of both tiles against 2200 of tensor work (59 % busy); issue slots are 57 %
// full. What it does not spend its time on alone: without the exponentials 4.5 % less,
// without the values' conversion 6.5 %, with half of each product 13 %.
// Slower: scores of 64 tokens at a time, issued as soon as their columns are free (1744
// us: the query operand is read twice as often); a second warp issuing products, one a
// tile (1773); scalar instead of paired arithmetic (1612 against 1563); a softmax that
// takes the last chunk's maximum before it has its own (2001 against 1582).
//
// Two builds share the code. PAIR: two adjacent query tiles share the K/V stream; one
// tile's softmax runs while the tensor core works on the other. Otherwise one tile,
// whose even and odd chunks go to the two softmax groups, each with its own maximum,
// sum and O, added at the end: for sequences of one tile and for calls of few
// blocks, whose key range may then be cut over several blocks too (splits; partials
// and merge as in pa_prefill_1t.cu).
//
// A tile's next scores take the tensor memory that its weights are in, and their product is
// issued right behind the value product that reads those. That rests on one thread's
// products of one CTA group being carried out in the order of issue, as in the bf16
// kernels, here for two kinds of them; the instruction set states that order for products
// of one accumulator and shape, and this use of it is held to equal bits over repeated
// prompts by tests. A wait between the two would leave the tensor core idle from the end
// of each value product until its commit had been seen, twice a chunk.
//
// Warps:
//   * 0-7, 8-15 (softmax groups): two threads a row, 64 of a chunk's 128 scores each;
//     they first turn the query rows into hi and lo;
//   * 16, 18: tiled bulk tensor copies of the K and V codes; 17: issues the products;
//     19: the scales of a chunk's pages, by table entry, into shared memory;
//   * 20-23: values' codes to f16; rows behind the last token become zeros.
// Every mbarrier wait is bounded. A role that gives up raises a shared abort flag
// (and PA_DEVERR_TIMEOUT); the others see it in their own waits. Before the block
// leaves, the copy warps wait (bounded) for their copies in flight, the MMA thread
// for its products, and the block frees its tensor memory.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_q8.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;      // M: query rows per tile
constexpr int kChunk = 128;     // tokens per chunk
constexpr int kD = 128;         // head dimension
constexpr int kGroupThreads = 2 * kRows;             // softmax threads of a group: two per row
constexpr int kSoftmaxThreads = 2 * kGroupThreads;
constexpr int kWarpK = kSoftmaxThreads / 32;         // warp 16
constexpr int kWarpMma = kWarpK + 1;
constexpr int kWarpV = kWarpMma + 1;
constexpr int kWarpScale = kWarpV + 1;
constexpr int kWarpConvert = kWarpScale + 1;         // and the three after it
constexpr int kConvertThreads = 128;
constexpr int kThreads = kSoftmaxThreads + 128 + kConvertThreads;
constexpr int kSortMax = 256;   // sequences ordered by length up to this batch size
constexpr uint32_t kTmemCols = 512;
// Tensor-memory columns: S of group t (128; W_t over its first 64), then O of group t.
__host__ __device__ constexpr uint32_t col_s(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * t; }
constexpr float kRaise = 8.f;   // raise the reference maximum only beyond this
constexpr float kBias = 7.f;    // weights times 2^7
// Registers a thread (setmaxnreg): what the launch has, and each role's share of it.
constexpr int kRegsLaunch = 80, kRegsSoftmax = 104, kRegsService = 32, kRegsConvert = 32;
static_assert(kSoftmaxThreads * kRegsSoftmax + 128 * kRegsService + kConvertThreads * kRegsConvert <=
                  kThreads * kRegsLaunch, "register shares");

// Shared-memory layout (byte offsets from a 1024-aligned base).
constexpr uint32_t kCodes = kChunk * kD;              // a chunk's codes: 128 rows x 128 B
constexpr uint32_t kTileQ = 2 * kRows * kD;           // hi, then lo: 128 rows x 128 B each
constexpr uint32_t kHalfV = kChunk * 128;             // 64 columns of a chunk in f16
constexpr uint32_t kStageV16 = 2 * kHalfV;
constexpr int kStagesV16 = 2;
template <bool PAIR>
struct Layout {
    static constexpr int kStagesK = PAIR ? 3 : 4;
    static constexpr int kStagesV = PAIR ? 2 : 3;
    static constexpr uint32_t kOffQ = 0;
    static constexpr uint32_t kOffK = kOffQ + (PAIR ? 2 : 1) * kTileQ;
    static constexpr uint32_t kOffV = kOffK + kStagesK * kCodes;
    static constexpr uint32_t kOffV16 = kOffV + kStagesV * kCodes;
    static constexpr uint32_t kOffBar = kOffV16 + kStagesV16 * kStageV16;
    // mbarriers (8 bytes each) and slots, at kOffBar + ...
    static constexpr uint32_t kKFull = 0;
    static constexpr uint32_t kKEmpty = kKFull + 8 * kStagesK;
    static constexpr uint32_t kVFull = kKEmpty + 8 * kStagesK;
    static constexpr uint32_t kVEmpty = kVFull + 8 * kStagesV;     // kConvertThreads arrivals
    static constexpr uint32_t kV16Full = kVEmpty + 8 * kStagesV;   // kConvertThreads arrivals
    static constexpr uint32_t kV16Empty = kV16Full + 16;           // value products of a chunk done
    static constexpr uint32_t kScale = kV16Empty + 16;             // [chunk % 2] scales written
    static constexpr uint32_t kS = kScale + 16;                    // [group] scores ready
    static constexpr uint32_t kP = kS + 16;                        // [part][group] weights stored, kGroupThreads arrivals
    static constexpr uint32_t kO = kP + 32;                        // the last value product done
    static constexpr uint32_t kQ = kO + 8;                         // queries written, kSoftmaxThreads arrivals
    static constexpr uint32_t kDrain = kQ + 8;
    static constexpr uint32_t kProbe = kDrain + 8;                 // nothing completes it
    static constexpr uint32_t kTmem = kProbe + 8;
    static constexpr uint32_t kAbort = kTmem + 4;
    static constexpr uint32_t kSeq = kAbort + 4;
    // Scales of a chunk's pages, [chunk % 2][page] (score factor, log2 vs, 2^24 / vs, -).
    static constexpr uint32_t kOffScale = kOffBar + 256;
    // The lengths of the ordering, then (maximum, sum) of group 1's rows.
    static constexpr uint32_t kOffRows = kOffScale + 2 * 8 * 16;
    static constexpr uint32_t kBytes = 1024 + kOffRows + 8 * kRows;
    static_assert(kSeq + 4 <= 256 && 8 * kRows >= 4 * kSortMax, "areas overlap");
    static_assert(kBytes <= 227 * 1024 && 2 * kBytes > 228 * 1024,
                  "one block per SM: it holds all 512 tensor-memory columns");
};

struct Q8PrefillArgs {
    const uint16_t* q;        // [T][Hq][D] bf16
    const float *k_scale, *v_scale;
    const int32_t* q_start;   // [B + 1]
    const int32_t* tables;
    const int32_t* seq_lens;
    void* out;                // [T][Hq][D]
    int* err;
    int B, Hq, Hkv, g, Qb;    // Qb = queries per tile = 128 / g
    int num_q, max_q;
    int max_blocks, num_blocks, max_seq_len;
    float scale_log2;
    int out_bf16, probe_wait;
    int splits, tiles, num_parts;   // key split of the one-tile build
    float* part;
};

__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
}

// A thread's 64 values of O times alpha.
__device__ __noinline__ void rescale(uint32_t o_addr, float alpha) {
#pragma unroll 1
    for (int piece = 0; piece < 8; ++piece) {
        float o[8];
        tc::ld16x2_8<64>(o_addr + 8 * piece, o);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= alpha;
        tc::st16x2_8<64>(o_addr + 8 * piece, o);
    }
}

// 32 elements of an output row from element d0 on.
__device__ __forceinline__ void write_row(const Q8PrefillArgs& a, size_t row, const float (&v)[32], float inv, int d0) {
    if (a.out_bf16) {
        uint16_t* o = static_cast<uint16_t*>(a.out) + row * kD + d0;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
            *reinterpret_cast<uint4*>(o + i) =
                make_uint4(pack_bf16x2(v[i] * inv, v[i + 1] * inv), pack_bf16x2(v[i + 2] * inv, v[i + 3] * inv),
                           pack_bf16x2(v[i + 4] * inv, v[i + 5] * inv), pack_bf16x2(v[i + 6] * inv, v[i + 7] * inv));
    } else {
        float* o = static_cast<float*>(a.out) + row * kD + d0;
#pragma unroll
        for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(o + i) =
                make_float4(v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv);
    }
}

// Zeroes output rows [r0, r1) x query heads [h0, h0 + g), the block's threads in turn.
__device__ void zero_rows(const Q8PrefillArgs& a, int64_t r0, int64_t r1, int h0, int tid) {
    const int64_t per_row = static_cast<int64_t>(a.g) * kD;
    for (int64_t i = tid; i < (r1 - r0) * per_row; i += kThreads) {
        const int64_t r = r0 + i / per_row;
        const size_t at = (static_cast<size_t>(r) * a.Hq + h0) * kD + static_cast<size_t>(i % per_row);
        if (a.out_bf16) static_cast<uint16_t*>(a.out)[at] = 0;
        else static_cast<float*>(a.out)[at] = 0.f;
    }
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int BS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const Q8PrefillArgs a) {
    using M = Layout<PAIR>;
    constexpr int kPages = kChunk / BS, kHalfPages = kPages / 2;  // of a chunk, of a thread's 64 scores
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + M::kOffBar;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + M::kOffBar + M::kAbort);
    int* seq_slot = reinterpret_cast<int*>(gbase + M::kOffBar + M::kSeq);

    // The sequence of this block: blockIdx.z is its rank by length (longest first, ties
    // by index) when the batch is small enough to rank here.
    int b = blockIdx.z;
    if (a.B <= kSortMax) {
        int* lens = reinterpret_cast<int*>(gbase + M::kOffRows);
        for (int i = tid; i < a.B; i += kThreads) lens[i] = a.seq_lens[i];
        __syncthreads();
        for (int i = tid; i < a.B; i += kThreads) {
            const int li = lens[i];
            int r = 0;
            for (int j = 0; j < a.B; ++j) {
                const int lj = lens[j];
                r += (lj > li) || (lj == li && j < i);
            }
            if (r == static_cast<int>(blockIdx.z)) *seq_slot = i;
        }
        __syncthreads();
        b = *seq_slot;
    }
    const int h = blockIdx.y;
    const int L = a.seq_lens[b];
    {
        const int64_t q64 = a.q_start[b], n64 = static_cast<int64_t>(a.q_start[b + 1]) - q64;
        if (n64 == 0) return;  // a request without queries in this step
        if (n64 < 0 || n64 > a.max_q || L < n64 || L > min(a.max_seq_len, a.max_blocks * BS) || q64 < 0 ||
            q64 + n64 > a.num_q) {
            if (blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(a.err, kErrSeqLen);
            if (blockIdx.x == 0)
                zero_rows(a, q64 > 0 ? q64 : 0, n64 > 0 ? (q64 + n64 < a.num_q ? q64 + n64 : a.num_q) : 0, h * a.g,
                          tid);
            return;
        }
    }
    const int qs = a.q_start[b];
    const int n = a.q_start[b + 1] - qs;
    const int per_block = PAIR ? 2 * a.Qb : a.Qb;
    const int split = PAIR ? 0 : blockIdx.x % a.splits;
    // The sequence's last tiles first: they have the most chunks.
    const int tile = (n + per_block - 1) / per_block - 1 - (PAIR ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) / a.splits);
    if (tile < 0) return;
    const int q0 = tile * per_block;
    const int nq0 = min(a.Qb, n - q0);
    const int nq1 = PAIR ? max(0, min(a.Qb, n - q0 - a.Qb)) : 0;
    const bool two = !PAIR || nq1 > 0;  // whether group 1 has work
    const int ntok = L - n + q0 + (nq1 > 0 ? a.Qb + nq1 : nq0);  // tokens the last row sees
    const int nc = (ntok + kChunk - 1) / kChunk;
    const int nb = (ntok + BS - 1) / BS;
    const int32_t* table = a.tables + static_cast<size_t>(b) * a.max_blocks;
    // This block's chunks: c_beg .. c_beg + nk - 1. Stages, phases and groups count k = c - c_beg.
    const int per = PAIR ? nc : (nc + a.splits - 1) / a.splits;
    const int c_beg = PAIR ? 0 : min(nc, split * per);
    const int nk = PAIR ? nc : min(nc, c_beg + per) - c_beg;
    const bool partial = !PAIR && a.splits > 1;
    const size_t pidx = ((static_cast<size_t>(b) * a.Hkv + h) * a.tiles + tile) * a.splits + split;
    float* part_o = partial ? a.part + pidx * kRows * kD : nullptr;
    float* part_ml = partial ? a.part + static_cast<size_t>(a.num_parts) * kRows * kD + pidx * kRows * 2 : nullptr;
    if (nk == 0) {  // a split past a short sequence's end: an empty partial
        if (tid < kRows) {
            part_ml[2 * tid] = -INFINITY;
            part_ml[2 * tid + 1] = 0.f;
        }
        return;
    }

    // This thread's query row (softmax warps): group t, row r of its tile, and which
    // half of the row's 128 columns it holds. Each warp lies within its tensor-memory
    // lane quarter; threads i and i + 16 share a row.
    const int t = (tid / kGroupThreads) & 1;
    const int quarter = warp & 3, sub16 = (warp >> 2) & 1, half = lane >> 4;
    const int row = 32 * quarter + 16 * sub16 + (lane & 15);
    const bool softmax = tid < kSoftmaxThreads;
    const int qi = row / a.g, qj = row - qi * a.g;
    const bool row_valid = softmax && qi < (PAIR && t ? nq1 : nq0);
    const size_t out_row = (static_cast<size_t>(qs) + q0 + (PAIR ? t * a.Qb : 0) + qi) * a.Hq + h * a.g + qj;

    if (tid == 0) {
        for (int s = 0; s < M::kStagesK; ++s) {
            mbar_init(bars + M::kKFull + 8 * s, 1);
            mbar_init(bars + M::kKEmpty + 8 * s, 1);
        }
        for (int s = 0; s < M::kStagesV; ++s) {
            mbar_init(bars + M::kVFull + 8 * s, 1);
            mbar_init(bars + M::kVEmpty + 8 * s, kConvertThreads);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bars + M::kV16Full + 8 * s, kConvertThreads);
            mbar_init(bars + M::kV16Empty + 8 * s, 1);
            mbar_init(bars + M::kScale + 8 * s, 1);
            mbar_init(bars + M::kS + 8 * s, 1);
            mbar_init(bars + M::kP + 8 * s, kGroupThreads);
            mbar_init(bars + M::kP + 16 + 8 * s, kGroupThreads);
        }
        mbar_init(bars + M::kO, 1);
        mbar_init(bars + M::kQ, kSoftmaxThreads);
        mbar_init(bars + M::kDrain, 1);
        mbar_init(bars + M::kProbe, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    // The table entries this block reads, validated once.
    bool bad = false;
    for (int i = tid; i < nb; i += kThreads) {
        const int p = table[i];
        bad |= p < 0 || p >= a.num_blocks;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(a.err, kErrTable);
        if (row_valid && (PAIR || t == 0)) {
            float z[32] = {};
            write_row(a, out_row, z, 0.f, 64 * half);
            write_row(a, out_row, z, 0.f, 64 * half + 32);
        }
        if (partial && tid < kRows) part_ml[2 * tid] = NAN;  // the merge writes zeros too
        return;
    }
    // Tensor memory, for the softmax and MMA warps, which meet on a barrier of their own.
    uint32_t tmem = 0;
    if (warp <= kWarpMma && warp != kWarpK) {
        if (warp == kWarpMma) {
            tc::alloc(bars + M::kTmem, kTmemCols);
            tc::relinquish();
        }
        tc::fence_before_sync();
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads + 32) : "memory");
        tc::fence_after_sync();
        tmem = *reinterpret_cast<volatile uint32_t*>(gbase + M::kOffBar + M::kTmem);
    }

    if (softmax) {
        // ------------------------------------------------------------ softmax (group t)
        regs_inc<kRegsSoftmax>();
        // The query row as hi + lo, in the swizzled K-major layout of the score
        // products' A operand. In the one-tile build both groups read the rows and
        // group 0 writes hi, group 1 lo.
        float sq;  // score factor of the row: its power of two
        {
            const uint4* src = reinterpret_cast<const uint4*>(a.q + out_row * kD + 64 * half);
            uint4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = row_valid ? src[i] : make_uint4(0, 0, 0, 0);
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = fabsf(bf16_lo(u[e])), y = fabsf(bf16_hi(u[e]));
                    most = fmaxf(most, fmaxf(x <= FLT_MAX ? x : 0.f, y <= FLT_MAX ? y : 0.f));
                }
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
            sq = q8::scale_for(most, 1u);  // down to 2^-126: rows of any size keep the same bits
            const float inv = 1.f / sq;    // a power of two
            const uint32_t dst = base + M::kOffQ + (PAIR ? t * kTileQ : 0) + row * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 v = w[2 * i + (e >> 1)];
                    const uint32_t u0 = e & 1 ? v.z : v.x, u1 = e & 1 ? v.w : v.y;
                    // Infinities become NaN, as e4m3 has none.
                    float x[4] = {bf16_lo(u0), bf16_hi(u0), bf16_lo(u1), bf16_hi(u1)};
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = fmaf(x[k], 0.f, x[k] * inv);
                    hi[e] = q8::from_f32x4(x[0], x[1], x[2], x[3]);
                    const float2 p = q8::f16x2_split(q8::to_f16x2(hi[e])), r = q8::f16x2_split(q8::hi_to_f16x2(hi[e]));
                    lo[e] = q8::from_f32x4(x[0] - p.x, x[1] - p.y, x[2] - r.x, x[3] - r.y);
                }
                const uint32_t at = dst + (((4 * half + i) ^ (row & 7)) << 4);
                if (PAIR || t == 0) st_shared_v4(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                if (PAIR || t == 1) st_shared_v4(at + kRows * 128, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
            fence_proxy_async_smem();
            mbar_arrive(bars + M::kQ);
        }
        const uint32_t lane_base = static_cast<uint32_t>(32 * quarter + 16 * sub16) << 16;
        const uint32_t s_addr = tmem + lane_base + col_s(t);
        const uint32_t o_addr = tmem + lane_base + col_o(t);
        const int pos_r = L - n + q0 + (PAIR ? t * a.Qb : 0) + qi;  // last token this row sees
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        const bool busy = t == 0 || two;
        for (int k = PAIR ? 0 : t, i = 0; k < nk && busy; k += PAIR ? 1 : 2, ++i) {
            const int c = c_beg + k;
            // The factors of this half's pages, before the scores are waited for.
            ok = __all_sync(0xffffffffu, wait_role(bars + M::kScale + 8 * (k & 1), (k >> 1) & 1, abort_flag, a.err));
            if (!ok) break;
            const float4* const page = reinterpret_cast<const float4*>(gbase + M::kOffScale) + (k & 1) * 8 + half * kHalfPages;
            float fac[kHalfPages], off[kHalfPages];
#pragma unroll
            for (int p = 0; p < kHalfPages; ++p) {
                const float2 f = *reinterpret_cast<const float2*>(page + p);
                fac[p] = fmaxf(f.x * sq, FLT_MIN);  // never 0: masked scores are -inf
                off[p] = f.y;
            }
            // Scores done; their commit also covers the group's value product before.
            ok = __all_sync(0xffffffffu, wait_role(bars + M::kS + 8 * t, i & 1, abort_flag, a.err));
            if (!ok) break;
            tc::fence_after_sync();
            // The scores' maximum, weights and sum. FAR: value scales far apart (pa_q8.cuh).
            auto weights = [&](auto far) {
                constexpr bool FAR = decltype(far)::value;
                float sv[kChunk / 2];
                tc::ld16x2_32<64>(s_addr, *reinterpret_cast<float(*)[32]>(sv));
                tc::ld16x2_32<64>(s_addr + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
                tc::wait_ld();
                // Causal mask by predicate; the warp skips it when no row needs it. (Rows
                // past the tile's queries are never stored.)
                if (__any_sync(0xffffffffu, row_valid && c * kChunk + kChunk - 1 > pos_r)) {
                    const int last = pos_r - (c * kChunk + 64 * half);
#pragma unroll
                    for (int j = 0; j < kChunk / 2; ++j) sv[j] = j <= last ? sv[j] : -INFINITY;
                }
                // Row maximum in the log2 domain, page by page (factors are positive), then
                // the partner's half.
                float mp[kHalfPages][2];
#pragma unroll
                for (int p = 0; p < kHalfPages; ++p) {
                    mp[p][0] = fmaxf(sv[p * BS], sv[p * BS + 1]);
                    mp[p][1] = fmaxf(sv[p * BS + 2], sv[p * BS + 3]);
                }
#pragma unroll
                for (int j = 4; j < BS; j += 4)
#pragma unroll
                    for (int p = 0; p < kHalfPages; ++p) {
                        mp[p][0] = max3(mp[p][0], sv[p * BS + j], sv[p * BS + j + 1]);
                        mp[p][1] = max3(mp[p][1], sv[p * BS + j + 2], sv[p * BS + j + 3]);
                    }
#pragma unroll
                for (int p = 0; p < kHalfPages; ++p) mp[p][0] = fmaf(fmaxf(mp[p][0], mp[p][1]), fac[p], off[p]);
                float mx = fmaxf(mp[0][0], mp[1][0]);
                if constexpr (kHalfPages == 4) mx = max3(mx, mp[2][0], mp[3][0]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                float alpha = 1.f;
                if (mx > m + kRaise) {
                    alpha = fast_exp2(m - mx);  // 0 while m is still -inf
                    if constexpr (FAR) l = q8::times_exp2(l, m - mx);
                    else l *= alpha;
                    m = mx;
                }
                const float m_use = (m == -INFINITY ? 0.f : m) - kBias;
                if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) rescale(o_addr, alpha);
                // W = 2^(s' - m) (f16 pairs) over columns 32 half .. of the row; the arguments
                // and sums two at a time, a page's sum times 1 / vs into l. In two parts, of 32
                // of each half's 64 tokens: the first part's product runs while the second is
                // computed.
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t pw[16];
#pragma unroll
                    for (int p = 0; p < 32 / BS; ++p) {
                        const int pg = h2 * (32 / BS) + p;
                        const uint64_t sc2 = f32x2(fac[pg], fac[pg]), of2 = f32x2(off[pg] - m_use, off[pg] - m_use);
                        uint64_t sum[2];
#pragma unroll
                        for (int j = 0; j < BS / 2; ++j) {
                            const int e = pg * BS + 2 * j;
                            const float2 x = f32x2_split(fma_f32x2(f32x2(sv[e], sv[e + 1]), sc2, of2));
                            const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                            sum[j & 1] = j < 2 ? f32x2(p0, p1) : add_f32x2(sum[j & 1], f32x2(p0, p1));
                            pw[p * (BS / 2) + j] = pack_f16x2(p0, p1);
                        }
                        const float2 s2 = f32x2_split(add_f32x2(sum[0], sum[1]));
                        if constexpr (FAR) {
#pragma unroll
                            for (int j = 0; j < BS; ++j) l += fast_exp2(fmaf(sv[pg * BS + j], fac[pg], q8::kSumBias - m_use));
                        } else {
                            l = fmaf(s2.x + s2.y, page[pg].z, l);
                        }
                    }
                    tc::st16x2_16u<32>(s_addr + 16 * h2, pw);
                    tc::wait_st();
                    tc::fence_before_sync();
                    mbar_arrive(bars + M::kP + 16 * h2 + 8 * t);
                }
            };
            if (__float_as_uint(off[0]) & 1u) weights(std::true_type());
            else weights(std::false_type());
        }
        // Epilogue.
        bool fine = ok && busy && __all_sync(0xffffffffu, wait_role(bars + M::kO, 0, abort_flag, a.err));
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if constexpr (PAIR) {
            if (fine) {
                tc::fence_after_sync();
                const float inv = q8::kSumFactor / l;
#pragma unroll
                for (int piece = 0; piece < 2; ++piece) {
                    float o[32];
                    tc::ld16x2_32<64>(o_addr + 32 * piece, o);
                    tc::wait_ld();
                    if (row_valid) write_row(a, out_row, o, inv, 64 * half + 32 * piece);
                }
            }
        } else {
            // Both groups' maxima, sums and O of the row; group t writes 32 of the 64
            // columns of each thread half.
            float2* rows = reinterpret_cast<float2*>(gbase + M::kOffRows);
            asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
            if (t == 1 && half == 0) rows[row] = make_float2(m, l);
            asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
            const float2 r1 = rows[row];
            asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
            if (t == 0 && half == 0) rows[row] = make_float2(m, l);
            asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
            const float2 r0 = rows[row];
            if (fine && !*abort_flag) {
                tc::fence_after_sync();
                const float mt = fmaxf(r0.x, r1.x), mu = mt == -INFINITY ? 0.f : mt;
                const float f0 = fast_exp2(r0.x - mu), f1 = fast_exp2(r1.x - mu);  // 0 without a score
                // (Sums without a score that is a number: 0, or NaN, which shows.)
                const float lt = (r0.x == -INFINITY ? r0.y : q8::times_exp2(r0.y, r0.x - mu)) +
                                 (r1.x == -INFINITY ? r1.y : q8::times_exp2(r1.y, r1.x - mu));
                const uint32_t at = tmem + lane_base + 32 * t;
                float o[32];
                tc::ld16x2_32<64>(at + col_o(0), o);
                tc::wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= f0;
                if (nk > 1) {
#pragma unroll
                    for (int piece = 0; piece < 4; ++piece) {
                        float x[8];
                        tc::ld16x2_8<64>(at + col_o(1) + 8 * piece, x);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[8 * piece + j] = fmaf(x[j], f1, o[8 * piece + j]);
                    }
                }
                if (row_valid) {
                    if (!partial) {
                        write_row(a, out_row, o, q8::kSumFactor / lt, 64 * half + 32 * t);
                    } else {
                        float* dst = part_o + static_cast<size_t>(row) * kD + 64 * half + 32 * t;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4*>(dst + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                        if (t == 0 && half == 0) {
                            part_ml[2 * row] = mt;
                            part_ml[2 * row + 1] = lt * (1.f / q8::kSumFactor);
                        }
                    }
                }
            }
        }
    } else if (warp < kWarpConvert) {
        regs_dec<kRegsService>();
        if (warp == kWarpK || warp == kWarpV) {
            // -------------------------------------------------------- copies of codes
            // (The whole warp, one thread issuing: addresses stay in uniform registers.)
            const bool is_k = warp == kWarpK;
            const uint32_t one = elect_one();
            const int nst = is_k ? M::kStagesK : M::kStagesV;
            const uint32_t full = bars + (is_k ? M::kKFull : M::kVFull);
            const uint32_t empty = bars + (is_k ? M::kKEmpty : M::kVEmpty);
            const uint32_t ring = base + (is_k ? M::kOffK : M::kOffV);
            const CUtensorMap* map = is_k ? &kmap : &vmap;
            // Lane j: the entry of page j of a chunk, loaded one chunk ahead.
            auto entry = [&](int c) {
                const int p = c * kPages + lane;
                return lane < kPages && p < nb ? table[p] : 0;
            };
            int pg = entry(c_beg), issued = 0;
            for (int k = 0; k < nk; ++k) {
                const int c = c_beg + k, s = k % nst;
                const bool ok = k < nst || wait_role(empty + 8 * s, ((k / nst) - 1) & 1, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) break;
                const int np = min(kPages, nb - c * kPages);
                const uint32_t bar = full + 8 * s, stage = ring + s * kCodes;
                if (one) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np) * BS * kD);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kPages; ++j)
                    tma_load_3d_if(j < np ? one : 0u, stage + j * BS * kD, map, 0, 0,
                                   __shfl_sync(0xffffffffu, pg, j) * a.Hkv + h, bar);
                issued = k + 1;
                pg = entry(c + 1);
            }
            // Copies still in flight land before the block leaves.
            for (int k = max(0, issued - nst); k < issued; ++k)
                mbar_wait_bounded(full + 8 * (k % nst), (k / nst) & 1, kWaitLimitNs);
        } else if (warp == kWarpMma) {
            // -------------------------------------------------------- products
            // (The whole warp, one thread issuing.)
            {
                const uint32_t one = elect_one();
                const uint32_t hi = static_cast<uint32_t>(tc::smem_desc(base, 16, 1024) >> 32);
                const uint32_t lo_q = tc::desc_lo(base + M::kOffQ, 16);
                const uint32_t lo_k = tc::desc_lo(base + M::kOffK, 16);
                const uint32_t lo_v = tc::desc_lo(base + M::kOffV16, kHalfV);
                auto issue_s = [&](int u, int k) {
                    const uint32_t a0 = lo_q + (PAIR ? u * (kTileQ >> 4) : 0);
                    const uint32_t b0 = lo_k + (k % M::kStagesK) * (kCodes >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // 32 of hi's 128, then of lo's
                        tc::mma_f8_lo_if(one, tmem + col_s(u), a0 + (kk >> 2) * ((kRows * 128) >> 4) + (kk & 3) * 2,
                                      b0 + (kk & 3) * 2, hi, tc::idesc_e4m3_f32(kRows, kChunk), kk > 0);
                    tc::commit_if(one, bars + M::kS + 8 * u);
                };
                // Part p of W: 32 of each half's 64 tokens.
                auto issue_pv = [&](int u, int k, bool add, int p) {
                    const uint32_t b0 = lo_v + (k % kStagesV16) * (kStageV16 >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 16 tokens = 8 columns of W
                        const int kk = 4 * (i >> 1) + 2 * p + (i & 1);
                        tc::mma_bf16_ts_if(one, tmem + col_o(u), tmem + col_s(u) + kk * 8, b0 + kk * (2048 >> 4), hi,
                                        tc::idesc_f16_f32(kRows, kD, false, true), add || i > 0);
                    }
                };
                auto wait = [&](uint32_t bar, int phase) {
                    return __all_sync(0xffffffffu, wait_role(bar, phase & 1, abort_flag, a.err)) != 0;
                };
                auto k_full = [&](int k) { return wait(bars + M::kKFull + 8 * (k % M::kStagesK), k / M::kStagesK); };
                auto v_full = [&](int k) { return wait(bars + M::kV16Full + 8 * (k % 2), k / 2); };
                auto w_full = [&](int u, int phase, int p) { return wait(bars + M::kP + 16 * p + 8 * u, phase); };
                bool ok;
                if (a.probe_wait) {
                    // The wait-expiry probe: a bounded wait on a barrier nothing
                    // completes, then the abort every other role follows.
                    mbar_wait_bounded(bars + M::kProbe, 0, kProbeLimitNs);
                    *abort_flag = 1;
                    if (one) atomicOr(a.err, kErrTimeout);
                    ok = false;
                } else {
                    ok = wait(bars + M::kQ, 0);
                }
                if constexpr (PAIR) {
                    if (ok && (ok = k_full(0))) {
                        tc::fence_after_sync();
                        issue_s(0, 0);
                        if (two) issue_s(1, 0);
                        tc::commit_if(one, bars + M::kKEmpty);
                    }
                    for (int k = 0; k < nk && ok; ++k) {
                        const int k1 = k + 1;
                        // What is ready early is waited for first.
                        ok = v_full(k) && (k1 == nk || k_full(k1));
                        for (int u = 0; u < (two ? 2 : 1) && ok; ++u) {
                            if (!(ok = w_full(u, k, 0))) break;
                            tc::fence_after_sync();
                            issue_pv(u, k, k > 0, 0);
                            if (!(ok = w_full(u, k, 1))) break;
                            tc::fence_after_sync();
                            issue_pv(u, k, true, 1);
                            if (u == (two ? 1 : 0)) tc::commit_if(one, bars + M::kV16Empty + 8 * (k % 2));
                            if (k1 < nk) issue_s(u, k1);  // behind the value product, which reads W first (see above)
                        }
                        if (ok && k1 < nk) tc::commit_if(one, bars + M::kKEmpty + 8 * (k1 % M::kStagesK));
                    }
                } else {
                    for (int k = 0; k < min(2, nk) && ok; ++k) {
                        if (!(ok = k_full(k))) break;
                        tc::fence_after_sync();
                        issue_s(k, k);
                        tc::commit_if(one, bars + M::kKEmpty + 8 * k);
                    }
                    for (int k = 0; k < nk && ok; ++k) {
                        const int u = k & 1, k2 = k + 2;
                        ok = v_full(k) && w_full(u, k >> 1, 0);
                        if (!ok) break;
                        tc::fence_after_sync();
                        issue_pv(u, k, k > 1, 0);
                        if (!(ok = w_full(u, k >> 1, 1))) break;
                        tc::fence_after_sync();
                        issue_pv(u, k, true, 1);
                        tc::commit_if(one, bars + M::kV16Empty + 8 * u);
                        if (k2 < nk) {
                            if (!(ok = k_full(k2))) break;
                            tc::fence_after_sync();
                            issue_s(u, k2);
                            tc::commit_if(one, bars + M::kKEmpty + 8 * (k2 % M::kStagesK));
                        }
                    }
                }
                if (ok) tc::commit_if(one, bars + M::kO);
                if (*abort_flag) {
                    tc::commit_if(one, bars + M::kDrain);
                    mbar_wait_bounded(bars + M::kDrain, 0, kWaitLimitNs);
                }
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- scales
            // Lane j reads page j's through its table entry, a chunk ahead; the slot of
            // chunk k is free once the value products of chunk k - 2, whose weights
            // came after its softmax, are done.
            float ks = 1.f, vs = 1.f;
            float top = -INFINITY, bottom = INFINITY;  // log2 of the largest and smallest value scale so far
            auto load = [&](int c) {
                const int p = c * kPages + lane;
                ks = vs = 1.f;
                if (lane < kPages && p < nb) {
                    const size_t at = static_cast<size_t>(table[p]) * a.Hkv + h;
                    ks = a.k_scale[at];
                    vs = a.v_scale[at];
                }
            };
            load(c_beg);
            for (int k = 0; k < nk; ++k) {
                const float f = ks * a.scale_log2, lv = q8::log2_of(vs, ks);
                const bool here = lane < kPages && (c_beg + k) * kPages + lane < nb;
                float most = here ? lv : -INFINITY, least = here ? lv : INFINITY;
#pragma unroll
                for (int off = 4; off > 0; off >>= 1) {
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, off));
                }
                top = fmaxf(top, __shfl_sync(0xffffffffu, most, 0));
                bottom = fminf(bottom, __shfl_sync(0xffffffffu, least, 0));
                // Whether they are far apart (pa_q8.cuh) goes with every page of the chunk as the last bit of
                // its log2 vs (at most 2^-17 of it off): the softmax has no register to spare for a flag.
                const uint32_t far = top - bottom > q8::kFarApart ? 1u : 0u;
                const float iv = q8::kSumFactor / vs;
                if (k + 1 < nk) load(c_beg + k + 1);
                bool ok = k < 2 || wait_role(bars + M::kV16Empty + 8 * (k & 1), ((k >> 1) - 1) & 1, abort_flag, a.err);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane < kPages)
                    st_shared_v4(base + M::kOffScale + ((k & 1) * 8 + lane) * 16,
                                 make_uint4(__float_as_uint(f), (__float_as_uint(lv) & ~1u) | far, __float_as_uint(iv), 0));
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + M::kScale + 8 * (k & 1));
            }
        }
    } else {
        // ------------------------------------------------------------ values to f16
        // Eight 16-code vectors a thread and chunk, a warp 32 rows. Eight neighbouring
        // threads take 64 codes of row r and of row r ^ 5, whose swizzles differ in bits 0
        // and 2: no bank conflicts, neither in the codes nor in the halves.
        regs_dec<kRegsConvert>();
        const int cw = warp - kWarpConvert, ch = (lane & 3) + 4 * ((lane >> 3) & 1);
        const int r0 = lane >> 4 ^ (lane & 4 ? 5 : 0), hc = 2 * (lane & 3);
        const uint32_t from = base + M::kOffV + 32 * 128 * cw + r0 * 128 + ((ch ^ r0) << 4);
        const uint32_t to = base + M::kOffV16 + 32 * 128 * cw + (ch >> 2) * kHalfV + r0 * 128 + ((hc ^ r0) << 4);
        for (int k = 0; k < nk; ++k) {
            const int s = k % M::kStagesV, s16 = k % kStagesV16;
            const int valid = min(kChunk, ntok - (c_beg + k) * kChunk) - 32 * cw;  // of this warp's 32 rows
            bool ok = wait_role(bars + M::kVFull + 8 * s, (k / M::kStagesV) & 1, abort_flag, a.err) &&
                      (k < kStagesV16 ||
                       wait_role(bars + M::kV16Empty + 8 * s16, ((k / kStagesV16) - 1) & 1, abort_flag, a.err));
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t src = from + s * kCodes, dst = to + s16 * kStageV16;
            auto convert = [&](bool ragged) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // Rows 8 (i / 2) + r0 + 2 (i & 1): the swizzle of the odd ones is 2 further.
                    const uint32_t row = (i >> 1) * 1024, odd = i & 1;
                    uint4 w = lds_u128((odd ? (src ^ 32) + 256 : src) + row);
                    if (ragged && 8 * (i >> 1) + r0 + (odd ? 2 : 0) >= valid) w = make_uint4(0, 0, 0, 0);
                    const uint32_t at = (odd ? (dst ^ 32) + 256 : dst) + row;
                    st_shared_v4(at, make_uint4(q8::to_f16x2(w.x), q8::hi_to_f16x2(w.x), q8::to_f16x2(w.y), q8::hi_to_f16x2(w.y)));
                    st_shared_v4(at ^ 16, make_uint4(q8::to_f16x2(w.z), q8::hi_to_f16x2(w.z), q8::to_f16x2(w.w), q8::hi_to_f16x2(w.w)));
                }
            };
            if (valid >= 32)
                convert(false);
            else
                convert(true);
            fence_proxy_async_smem();
            mbar_arrive(bars + M::kV16Full + 8 * s16);
            mbar_arrive(bars + M::kVEmpty + 8 * s);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        tc::fence_after_sync();
        tc::dealloc(tmem, kTmemCols);
    }
}

}  // namespace

cudaError_t launch_prefill_q8(const CUtensorMap& kmap, const CUtensorMap& vmap, const void* q, int num_q,
                              const int32_t* q_start, const int32_t* tables, const int32_t* seq_lens,
                              const float* k_scale, const float* v_scale, void* out, int* err, int B, int Hq,
                              int Hkv, int max_blocks, int num_blocks, int max_seq_len, int max_q, float scale_log2,
                              int out_bf16, int block_size, bool pair, float* part, int splits, cudaStream_t stream) {
    Q8PrefillArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.q_start = q_start;
    a.tables = tables;
    a.seq_lens = seq_lens;
    a.out = out;
    a.err = err;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.Qb = kRows / a.g;
    a.num_q = num_q;
    a.max_q = max_q;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.max_seq_len = max_seq_len;
    a.scale_log2 = scale_log2;
    a.out_bf16 = out_bf16;
    a.probe_wait = wait_probe();
    // No sequence has more queries than the call has rows.
    const int64_t nq = std::min<int64_t>(max_q, num_q);
    const int64_t tiles = (nq + a.Qb - 1) / a.Qb;
    if (splits < 1 || (splits > 1 && (pair || !part))) return cudaErrorInvalidValue;
    a.splits = splits;
    a.tiles = static_cast<int>(tiles);
    a.num_parts = static_cast<int>(tiles * Hkv * B * splits);
    a.part = splits > 1 ? part : nullptr;
    const dim3 grid(static_cast<unsigned>(pair ? (tiles + 1) / 2 : tiles * splits), Hkv, B);
    auto launch = [&](auto kern, uint32_t bytes) {
        // For every call in the process: the build's own size, whatever the call's.
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
        if (e != cudaSuccess) return e;
        kern<<<grid, kThreads, bytes, stream>>>(kmap, vmap, a);
        return cudaGetLastError();
    };
    const cudaError_t e = pair ? launch(block_size == 16 ? prefill_q8_kernel<16, true> : prefill_q8_kernel<32, true>,
                                        Layout<true>::kBytes)
                               : launch(block_size == 16 ? prefill_q8_kernel<16, false> : prefill_q8_kernel<32, false>,
                                        Layout<false>::kBytes);
    if (e != cudaSuccess || splits == 1) return e;
    return launch_prefill_split_merge(part, a.tiles, splits, q_start, seq_lens, out, out_bf16, B, Hq, Hkv, num_q,
                                      std::min(max_seq_len, max_blocks * block_size), max_q, 1, stream);
}

}  // namespace pa
