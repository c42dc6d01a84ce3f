// Writing and reading a paged cache held in 8 bits: e4m3 codes with one scale for
// each block and kv head (pa_qk_rope_append_q8, pa_read_kv_q8).
//
// The unit of work is a block of the cache that holds rows of the call (an item,
// pa_q8.cuh): its scale depends on all of them, so one thread block (or a few,
// each with some of the heads) takes them together, and one warp all rows of a
// head. It takes the largest magnitude, settles the scale and writes the codes: no
// atomics, and no order of arrival in the result.
//   scale s = the smallest power of two with max |x| <= 448 s
// A power of two costs an e4m3 code no accuracy (its error is relative), makes
// code x scale exact in bf16, and lets a block's scale grow later without a second
// rounding of the codes that it holds already. A caller's own scale that is none stays
// while it is large enough; codes are then x (1 / s) in 32 bits rounded again, within
// 2^-22 of x of the quotient rounded once. Quotients rounded once there (a sticky last
// bit) took 2.4 to 8 % of every call's time, in the loop, as a loop of its own or in a
// function behind it: the kernel has no register to spare.
//
// The sines of a block's rows are computed once for all heads, into shared memory. A
// warp holds two steps of loads (8 rows at D = 128), turns them for the maximum, and
// reads and turns them again, from L1, for the codes.
//
// Measured (device time; the copy rate is 6.8 TB/s). Write and read-back of 41084
// prompt rows, 32 + 8 heads of 128 with norms: 227 us, 187 of them the write (0.90 GB
// of DRAM traffic, 4.9 TB/s): bound by issue slots (55 %, 2.3 instructions a clock) and
// the latency of loads with 22 warps an SM. 64 rows: 9.5 us (6.2 and 3.3), two launches
// and their chains of dependent lookups. 3875 rows, 48 + 12 heads of 64, half rotated: 24.3 us,
// 19.5 of them the write (65 MB, 3.4 TB/s: 139 blocks of the cache, in five parts each, are
// 1.5 rounds of the blocks that fit the SMs). Read-back of 89557 rows, 16 sequences: 86 us, 0.94 of
// the copy rate, in float32 142 us, 0.95, heads of 64 50 us, 0.81. Slower for the 41084 rows: two blocks an SM with more rows in
// registers (234 to 249 us), weights folded into a table of the turns (238 to 250
// us: the table's loads cost more than the products they save); asking for rows and
// positions before the table entry arrives (64 rows 16.6 us, 12.0 without at the time);
// steps without rows left out one by one, not two by two (9.2 us, but 230 against 228.5).
//
// Keys are turned in 32 bits: of 42 million codes about 75 differ from those of exact
// arithmetic, all of them values next to the middle of two codes (a plain form in 32
// bits has as many). A correctly rounded reciprocal root changes nothing (237 us); pairs
// within 64 units of a middle taken again in 64 bits leave 16, for 275 us and 16 us for
// 64 rows, and are not worth it: a code is off by up to 2^-4 either way.
#include <algorithm>
#include <cfloat>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_q8.cuh"
#include "pa_rope.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;        // warps a block
constexpr int kPairs = 64;       // pairs of a head at most
constexpr int kHeadBatch = 4;    // query heads whose loads are in flight together
constexpr int kSteps = 2;        // steps of rows of a kv head, the same

struct Q8WriteArgs : q8::RowArgs {
    const uint16_t *q, *k, *v;      // rows [T][H][D] bf16, row strides in elements
    uint16_t* q_out;
    uint8_t *kpool, *vpool;
    float *kscale, *vscale;
    const int32_t* positions;
    const uint16_t *q_weight, *k_weight;  // [D] or null
    int64_t q_stride, k_stride, v_stride, qo_stride;
    int Hq, Hkv, rot;
    float eps, amplitude;
    uint64_t turn[PA_ROPE_MAX_PAIRS];
};

// Infinities to NaN, as e4m3 has none: they count for nothing in a maximum and
// become the NaN code.
__device__ __forceinline__ uint64_t no_inf(uint64_t v) {
    float2 x = f32x2_split(v);
    if (fabsf(x.x) > FLT_MAX) x.x = __int_as_float(0x7fc00000);
    if (fabsf(x.y) > FLT_MAX) x.y = __int_as_float(0x7fc00000);
    return f32x2(x.x, x.y);
}

__device__ __forceinline__ float max_abs(float most, uint64_t v) {
    const float2 x = f32x2_split(v);
    return max3(most, fabsf(x.x), fabsf(x.y));  // passes over NaN
}

// The scale of a block whose rows of this call reach `most`; the codes of its
// off0 earlier tokens are brought to it. All lanes of the warp.
template <int D>
__device__ __forceinline__ float settle_scale(float most, int off0, float* scale, uint8_t* codes, int lane) {
    const float need = q8::scale_for(most);
    if (off0 == 0) {
        if (lane == 0) *scale = need;
        return need;
    }
    const float old = *scale;
    const float s = fmaxf(old, need);
    __syncwarp();
    if (s != old) {
        const float ratio = old / s;
        for (int i = lane; i < off0 * (D / 16); i += 32) {
            uint4 w = reinterpret_cast<uint4*>(codes)[i];
            uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = q8::f16x2_split(q8::to_f16x2(u[e])), b = q8::f16x2_split(q8::hi_to_f16x2(u[e]));
                u[e] = q8::from_f32x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
            }
            reinterpret_cast<uint4*>(codes)[i] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if (lane == 0) *scale = s;
    }
    return s;
}

template <int D, int BS, bool HALF>
__global__ void __launch_bounds__(32 * kWarps, 3) q8_write_kernel(const __grid_constant__ Q8WriteArgs a) {
    using P = Pairs<uint16_t, HALF>;
    constexpr int N = 8;              // elements a vector, pairs a thread
    constexpr int TPH = D / (2 * N);  // threads a head
    constexpr int RPW = 32 / TPH;     // rows a warp takes at a time: a step
    constexpr int STEPS = BS / RPW / 2 < kSteps ? BS / RPW / 2 : kSteps;  // steps whose rows a warp holds
    __shared__ __align__(16) float sines[BS][2][kPairs];  // [row][sin, cos][pair, in vectors of four]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    q8::Rows r;
    if (!q8::find_rows(a, blockIdx.x, blockIdx.x == 0 && blockIdx.y == 0, &r)) return;
    const int n = r.n;
    // Where pair p's sine lies: a thread's vectors of four pairs are next to its
    // neighbours' in memory (pairs 8 c .. 8 c + 7 of thread c with the half layout).
    auto place = [](int p) { return HALF ? (((p >> 2) & 1) * (kPairs / 8) + (p >> 3)) * 4 + (p & 3) : p; };
    if (a.rot) {
        const int half = a.rot / 2;
        for (int i = tid; i < n * half; i += 32 * kWarps) {
            const int row = i / half, p = i - row * half;
            const float2 sc = sin_cos(a.positions[r.row0 + row], a.turn[p]);
            sines[row][0][place(p)] = sc.x * a.amplitude;
            sines[row][1][place(p)] = sc.y * a.amplitude;
        }
        __syncthreads();
    }
    // This thread's row of a step, its two vectors of a head, and whether they turn.
    const int c = lane % TPH, sub = lane / TPH;
    int v0, v1;
    bool r0, r1;
    if constexpr (HALF) {
        const int n2 = a.rot / (2 * N);
        r0 = r1 = c < n2;
        v0 = r0 ? c : 2 * c;
        v1 = r0 ? n2 + c : 2 * c + 1;
    } else {
        v0 = c;
        v1 = c + TPH;
        r0 = v0 * N < a.rot;
        r1 = v1 * N < a.rot;
    }
    uint64_t sn[N / 2], cs[N / 2];
    auto load_sines = [&](int row) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int p = HALF ? c * N + 4 * j : (j ? v1 : v0) * (N / 2);
            const int at = place(p);
            const float4 s = *reinterpret_cast<const float4*>(&sines[row][0][at]);
            const float4 t = *reinterpret_cast<const float4*>(&sines[row][1][at]);
            sn[2 * j] = f32x2(s.x, s.y);
            sn[2 * j + 1] = f32x2(s.z, s.w);
            cs[2 * j] = f32x2(t.x, t.y);
            cs[2 * j + 1] = f32x2(t.z, t.w);
        }
    };
    // Mean square of the head whose vectors w0 and w1 are, as a factor.
    auto norm_of = [&](uint4 w0, uint4 w1) {
        uint64_t x1[N / 2], x2[N / 2];
        P::unpack(w0, w1, x1, x2);
        uint64_t s1 = f32x2(0.f, 0.f), s2 = s1;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            s1 = fma_f32x2(x1[i], x1[i], s1);
            s2 = fma_f32x2(x2[i], x2[i], s2);
        }
        const float2 s = f32x2_split(add_f32x2(s1, s2));
        float ss = s.x + s.y;
#pragma unroll
        for (int off = TPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        return rsqrtf(ss * (1.f / D) + a.eps);
    };
    auto turn = [&](uint4 w0, uint4 w1, bool weight, uint4 g0, uint4 g1, float rn, uint64_t (&x1)[N / 2],
                    uint64_t (&x2)[N / 2]) {
        P::unpack(w0, w1, x1, x2);
        if (weight) {
            const uint64_t rr = f32x2(rn, rn);
            uint64_t y1[N / 2], y2[N / 2];
            P::unpack(g0, g1, y1, y2);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                x1[i] = mul_f32x2(mul_f32x2(x1[i], rr), y1[i]);
                x2[i] = mul_f32x2(mul_f32x2(x2[i], rr), y2[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if (HALF || i < N / 4 ? r0 : r1) {
                const uint64_t z1 = x1[i], z2 = x2[i];
                const float2 m2 = f32x2_split(z2);
                x1[i] = fma_f32x2(f32x2(-m2.x, -m2.y), sn[i], mul_f32x2(z1, cs[i]));
                x2[i] = fma_f32x2(z1, sn[i], mul_f32x2(z2, cs[i]));
            }
        }
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto weights = [&](const uint16_t* w, uint4& g0, uint4& g1) {
        g0 = g1 = zero;
        if (w) {
            g0 = *reinterpret_cast<const uint4*>(w + v0 * N);
            g1 = *reinterpret_cast<const uint4*>(w + v1 * N);
        }
    };
    // Units: the kv heads' keys, their values, then batches of query heads of the
    // rows of one step.
    const int row_groups = (n + RPW - 1) / RPW, head_groups = (a.Hq + kHeadBatch - 1) / kHeadBatch;
    const int units = 2 * a.Hkv + row_groups * head_groups;
    for (int u = blockIdx.y * kWarps + warp; u < units; u += gridDim.y * kWarps) {
        if (u < a.Hkv) {  // keys of head u
            const uint16_t* src = a.k + static_cast<int64_t>(r.row0) * a.k_stride + u * D;
            uint4 w0[STEPS], w1[STEPS], g0, g1;
            auto load = [&](int first) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int row = (first + s) * RPW + sub;
                    w0[s] = w1[s] = zero;
                    if (row < n) {
                        w0[s] = *reinterpret_cast<const uint4*>(src + row * a.k_stride + v0 * N);
                        w1[s] = *reinterpret_cast<const uint4*>(src + row * a.k_stride + v1 * N);
                    }
                }
            };
            weights(a.k_weight, g0, g1);
            uint64_t x1[N / 2], x2[N / 2];
            float most;
            auto turned = [&](int first, int s, bool fix) {
                const float rn = a.k_weight ? norm_of(w0[s], w1[s]) : 1.f;
                if (a.rot) load_sines(min((first + s) * RPW + sub, n - 1));
                turn(w0[s], w1[s], a.k_weight != nullptr, g0, g1, rn, x1, x2);
                if (fix) {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        x1[i] = no_inf(x1[i]);
                        x2[i] = no_inf(x2[i]);
                    }
                }
            };
            bool fix = false;  // some element is infinite
            while (true) {
                most = 0.f;
#pragma unroll 1
                for (int f = 0; f < row_groups; f += STEPS) {
                    load(f);
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        turned(f, s, fix);
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) most = max_abs(max_abs(most, x1[i]), x2[i]);
                    }
                }
                if (fix || !__any_sync(0xffffffffu, most > FLT_MAX)) break;
                fix = true;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
            const size_t at = static_cast<size_t>(r.phys) * a.Hkv + u;
            uint8_t* codes = a.kpool + at * (BS * D);
            const float inv = 1.f / settle_scale<D>(most, r.off0, a.kscale + at, codes, lane);
#pragma unroll 1
            for (int f = 0; f < row_groups; f += STEPS) {
                load(f);  // again, from L1
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int row = (f + s) * RPW + sub;
                    turned(f, s, fix);
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint64_t s2 = f32x2(inv, inv);
                        const float2 xa = f32x2_split(mul_f32x2(x1[2 * i], s2));
                        const float2 xb = f32x2_split(mul_f32x2(x1[2 * i + 1], s2));
                        const float2 ya = f32x2_split(mul_f32x2(x2[2 * i], s2));
                        const float2 yb = f32x2_split(mul_f32x2(x2[2 * i + 1], s2));
                        if constexpr (HALF) {  // ends of the pairs: one vector each
                            o[i] = q8::from_f32x4(xa.x, xa.y, xb.x, xb.y);
                            o[2 + i] = q8::from_f32x4(ya.x, ya.y, yb.x, yb.y);
                        } else {               // whole pairs: vector i
                            o[2 * i] = q8::from_f32x4(xa.x, ya.x, xa.y, ya.y);
                            o[2 * i + 1] = q8::from_f32x4(xb.x, yb.x, xb.y, yb.y);
                        }
                    }
                    if (row < n) {
                        uint8_t* dst = codes + (r.off0 + row) * D;
                        *reinterpret_cast<uint2*>(dst + v0 * N) = make_uint2(o[0], o[1]);
                        *reinterpret_cast<uint2*>(dst + v1 * N) = make_uint2(o[2], o[3]);
                    }
                }
            }
        } else if (u < 2 * a.Hkv) {  // values of head u - Hkv, 16 neighbouring elements a thread
            const int h = u - a.Hkv;
            const uint16_t* src = a.v + static_cast<int64_t>(r.row0) * a.v_stride + h * D + c * 2 * N;
            uint4 w0[STEPS], w1[STEPS];
            auto load = [&](int first) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int row = (first + s) * RPW + sub;
                    w0[s] = w1[s] = zero;
                    if (row < n) {
                        w0[s] = *reinterpret_cast<const uint4*>(src + row * a.v_stride);
                        w1[s] = *reinterpret_cast<const uint4*>(src + row * a.v_stride + N);
                    }
                }
            };
            float most;
            bool fix = false;
            auto pair = [&](int s, int i) {  // elements 2 i and 2 i + 1 of the thread's 16
                const uint4& w = i < 4 ? w0[s] : w1[s];
                const uint32_t u = (i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w;
                const uint64_t v = f32x2(bf16_lo(u), bf16_hi(u));
                return fix ? no_inf(v) : v;
            };
            while (true) {
                most = 0.f;
#pragma unroll 1
                for (int f = 0; f < row_groups; f += STEPS) {
                    load(f);
#pragma unroll
                    for (int s = 0; s < STEPS; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i) most = max_abs(most, pair(s, i));
                }
                if (fix || !__any_sync(0xffffffffu, most > FLT_MAX)) break;
                fix = true;
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
            const size_t at = static_cast<size_t>(r.phys) * a.Hkv + h;
            uint8_t* codes = a.vpool + at * (BS * D);
            const float inv = 1.f / settle_scale<D>(most, r.off0, a.vscale + at, codes, lane);
#pragma unroll 1
            for (int f = 0; f < row_groups; f += STEPS) {
                load(f);  // again, from L1
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const int row = (f + s) * RPW + sub;
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = f32x2_split(mul_f32x2(pair(s, 2 * i), f32x2(inv, inv)));
                        const float2 y = f32x2_split(mul_f32x2(pair(s, 2 * i + 1), f32x2(inv, inv)));
                        o[i] = q8::from_f32x4(x.x, x.y, y.x, y.y);
                    }
                    if (row < n)
                        *reinterpret_cast<uint4*>(codes + (r.off0 + row) * D + c * 2 * N) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        } else {  // a batch of query heads
            const int i = u - 2 * a.Hkv, hg = i / row_groups;
            const int row = (i - hg * row_groups) * RPW + sub;
            const int h0 = hg * kHeadBatch, nh = min(kHeadBatch, a.Hq - h0);
            const uint16_t* src = a.q + (r.row0 + row) * a.q_stride + h0 * D;
            uint16_t* dst = a.q_out + (r.row0 + row) * a.qo_stride + h0 * D;
            uint4 w0[kHeadBatch], w1[kHeadBatch], g0, g1;
#pragma unroll
            for (int j = 0; j < kHeadBatch; ++j) {
                w0[j] = w1[j] = zero;
                if (row < n && j < nh) {
                    w0[j] = *reinterpret_cast<const uint4*>(src + j * D + v0 * N);
                    w1[j] = *reinterpret_cast<const uint4*>(src + j * D + v1 * N);
                }
            }
            weights(a.q_weight, g0, g1);
            if (a.rot) load_sines(min(row, n - 1));
#pragma unroll
            for (int j = 0; j < kHeadBatch; ++j) {
                const float rn = a.q_weight ? norm_of(w0[j], w1[j]) : 1.f;
                uint64_t x1[N / 2], x2[N / 2];
                turn(w0[j], w1[j], a.q_weight != nullptr, g0, g1, rn, x1, x2);
                uint4 o0, o1;
                P::pack(x1, x2, o0, o1);
                // A vector that is neither normalised nor rotated keeps its bits.
                if (!(a.q_weight || r0)) o0 = w0[j];
                if (!(a.q_weight || r1)) o1 = w1[j];
                if (row < n && j < nh) {
                    *reinterpret_cast<uint4*>(dst + j * D + v0 * N) = o0;
                    *reinterpret_cast<uint4*>(dst + j * D + v1 * N) = o1;
                }
            }
        }
    }
}

struct Q8ReadArgs : q8::RowArgs {
    const uint8_t *kpool, *vpool;
    const float *kscale, *vscale;
    void *k_out, *v_out;       // [T][Hkv][D]
    int Hkv;
};

// A warp takes the rows of one kv head of an item, K or V: a thread reads the codes
// of one 16-byte vector of the output.
template <int D, int BS, bool BF16>
__global__ void __launch_bounds__(32 * kWarps) q8_read_kernel(const __grid_constant__ Q8ReadArgs a) {
    constexpr int N = BF16 ? 8 : 4;      // elements a thread
    constexpr int TPR = D / N;           // threads a row
    constexpr int RPW = 32 / TPR;        // rows a warp takes at a time
    constexpr int BATCH = 8;             // loads in flight a thread
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch_dependents();
    q8::Rows r;
    if (!q8::find_rows(a, blockIdx.x, blockIdx.x == 0 && blockIdx.y == 0, &r)) return;
    const int c = lane % TPR, sub = lane / TPR;
    for (int u = blockIdx.y * kWarps + warp; u < 2 * a.Hkv; u += gridDim.y * kWarps) {
        const int h = u < a.Hkv ? u : u - a.Hkv;
        const size_t at = static_cast<size_t>(r.phys) * a.Hkv + h;
        const uint8_t* src = (u < a.Hkv ? a.kpool : a.vpool) + (at * BS + r.off0) * D + c * N;
        const float s = (u < a.Hkv ? a.kscale : a.vscale)[at];
        const size_t first = (static_cast<size_t>(r.row0) * a.Hkv + h) * D + c * N;
        const size_t pitch = static_cast<size_t>(a.Hkv) * D;
        for (int row0 = sub; row0 < r.n; row0 += RPW * BATCH) {
            uint2 w[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int row = row0 + j * RPW;
                w[j] = make_uint2(0, 0);
                if (row < r.n) {
                    if constexpr (BF16) w[j] = *reinterpret_cast<const uint2*>(src + row * D);
                    else w[j].x = *reinterpret_cast<const uint32_t*>(src + row * D);
                }
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int row = row0 + j * RPW;
                if (row >= r.n) break;
                float x[8];
#pragma unroll
                for (int e = 0; e < N / 4; ++e) {
                    const uint32_t u4 = e ? w[j].y : w[j].x;
                    const float2 lo = q8::f16x2_split(q8::to_f16x2(u4)), hi = q8::f16x2_split(q8::hi_to_f16x2(u4));
                    x[4 * e] = lo.x * s;
                    x[4 * e + 1] = lo.y * s;
                    x[4 * e + 2] = hi.x * s;
                    x[4 * e + 3] = hi.y * s;
                }
                void* out = u < a.Hkv ? a.k_out : a.v_out;
                if constexpr (BF16)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + first + row * pitch) =
                        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                   pack_bf16x2(x[6], x[7]));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(out) + first + row * pitch) =
                        make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
}

// The arguments that say which rows a call is about.
pa_status row_args(q8::RowArgs* a, const int32_t* q_start, const int32_t* tables, int max_blocks,
                   const int32_t* seq_lens, int B, int T, int block_size, int num_blocks, int Hkv, int* device_error) {
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (T < 0 || B < 0 || B > kMaxBatch || max_blocks < 1 || num_blocks < 1 || Hkv < 1 || Hkv > 65536 ||
        static_cast<int64_t>(num_blocks) * Hkv > INT32_MAX || static_cast<int64_t>(max_blocks) * block_size > INT32_MAX)
        return PA_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(q_start) | reinterpret_cast<uintptr_t>(tables) |
         reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(device_error)) & 3u)
        return PA_ERR_ALIGN;
    a->q_start = q_start;
    a->tables = tables;
    a->seq_lens = seq_lens;
    a->err = device_error;
    a->B = B;
    a->T = T;
    a->max_blocks = max_blocks;
    a->num_blocks = num_blocks;
    a->shift = block_size == 16 ? 4 : 5;
    return PA_OK;
}

// Items x parts: as many parts an item (thread blocks that share its heads) as
// fill the SMs, 32 warps each, when there are few items.
template <typename Args>
cudaError_t launch_rows(void (*fn)(Args), const Args& a, int units, cudaStream_t stream) {
    const int64_t items = (static_cast<int64_t>(a.T) >> a.shift) + 2LL * a.B;
    const int64_t full = (static_cast<int64_t>(a.T) >> a.shift) + a.B;  // that may hold rows, about
    const int64_t most = (units + kWarps - 1) / kWarps;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({most, kSms * 4 / full + 1, 64}));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items), static_cast<unsigned>(parts));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <int D, int BS>
void (*select_write(bool half))(Q8WriteArgs) {
    return half ? q8_write_kernel<D, BS, true> : q8_write_kernel<D, BS, false>;
}

template <int D, int BS>
void (*select_read(bool bf16))(Q8ReadArgs) {
    return bf16 ? q8_read_kernel<D, BS, true> : q8_read_kernel<D, BS, false>;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_qk_rope_append_q8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const int32_t* positions, const int32_t* q_start,
                               const int32_t* block_tables, int max_blocks, const int32_t* seq_lens, int B,
                               int num_rows, int Hq, int Hkv, int D, pa_dtype dtype, const void* q_weight,
                               const void* k_weight, float eps, const pa_rope* rope, void* q_out,
                               int64_t q_out_stride, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                               int block_size, int num_blocks, int* device_error, struct CUstream_st* stream) {
    if (!v || !q_start || !block_tables || !seq_lens || !k_pool || !v_pool || !k_scale || !v_scale) return PA_ERR_NULL;
    pa_status st = pa::rope_check(q, q_stride, k, k_stride, positions, num_rows, Hq, Hkv, D, dtype, q_weight, k_weight,
                                  eps, rope, q_out, q_out_stride);
    if (st != PA_OK) return st;
    if (dtype != PA_BF16) return PA_ERR_DTYPE;
    pa::Q8WriteArgs a{};
    st = pa::row_args(&a, q_start, block_tables, max_blocks, seq_lens, B, num_rows, block_size, num_blocks, Hkv,
                      device_error);
    if (st != PA_OK) return st;
    if (!pa::stride_ok(v_stride, Hkv, D, 2)) return PA_ERR_SHAPE;
    if (!pa::aligned16(v) || !pa::aligned16(k_pool) || !pa::aligned16(v_pool) ||
        ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u))
        return PA_ERR_ALIGN;
    if (num_rows == 0 || B == 0) return PA_OK;
    if (!a.err && pa::append_error_address(&a.err) != cudaSuccess) return PA_ERR_CUDA;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.kpool = static_cast<uint8_t*>(k_pool);
    a.vpool = static_cast<uint8_t*>(v_pool);
    a.kscale = k_scale;
    a.vscale = v_scale;
    a.positions = positions;
    a.q_weight = static_cast<const uint16_t*>(q_weight);
    a.k_weight = static_cast<const uint16_t*>(k_weight);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.eps = eps;
    if (rope) {
        a.rot = rope->rot_dim;
        a.amplitude = rope->amplitude;
        for (int i = 0; i < rope->rot_dim / 2; ++i) a.turn[i] = rope->turn[i];
    }
    const bool half = !rope || rope->layout == PA_ROPE_HALF;
    auto fn = D == 128 ? (block_size == 16 ? pa::select_write<128, 16>(half) : pa::select_write<128, 32>(half))
                       : (block_size == 16 ? pa::select_write<64, 16>(half) : pa::select_write<64, 32>(half));
    const int groups = (Hq + pa::kHeadBatch - 1) / pa::kHeadBatch;
    return pa::launch_rows(fn, a, 2 * Hkv + groups, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK
                                                                                                         : PA_ERR_CUDA;
}

pa_status pa_read_kv_q8(const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
                        const int32_t* block_tables, int max_blocks, const int32_t* seq_lens, const int32_t* q_start,
                        int B, int num_rows, int Hkv, int D, int block_size, int num_blocks, void* k_out, void* v_out,
                        pa_dtype out_dtype, int* device_error, struct CUstream_st* stream) {
    if (!k_pool || !v_pool || !k_scale || !v_scale || !block_tables || !seq_lens || !q_start || !k_out || !v_out)
        return PA_ERR_NULL;
    if (out_dtype != PA_F32 && out_dtype != PA_BF16) return PA_ERR_DTYPE;
    pa::Q8ReadArgs a{};
    const pa_status st = pa::row_args(&a, q_start, block_tables, max_blocks, seq_lens, B, num_rows, block_size,
                                      num_blocks, Hkv, device_error);
    if (st != PA_OK) return st;
    if (D != 64 && D != 128) return PA_ERR_SHAPE;
    if (!pa::aligned16(k_pool) || !pa::aligned16(v_pool) || !pa::aligned16(k_out) || !pa::aligned16(v_out) ||
        ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u))
        return PA_ERR_ALIGN;
    if (num_rows == 0 || B == 0) return PA_OK;
    if (!a.err && pa::append_error_address(&a.err) != cudaSuccess) return PA_ERR_CUDA;
    a.kpool = static_cast<const uint8_t*>(k_pool);
    a.vpool = static_cast<const uint8_t*>(v_pool);
    a.kscale = k_scale;
    a.vscale = v_scale;
    a.k_out = k_out;
    a.v_out = v_out;
    a.Hkv = Hkv;
    const bool bf16 = out_dtype == PA_BF16;
    auto fn = D == 128 ? (block_size == 16 ? pa::select_read<128, 16>(bf16) : pa::select_read<128, 32>(bf16))
                       : (block_size == 16 ? pa::select_read<64, 16>(bf16) : pa::select_read<64, 32>(bf16));
    return pa::launch_rows(fn, a, 2 * Hkv, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
