// Rotary positions, per-head norms and the cache write of a step's new rows.
//
// For every row t and head, with a_i = positions[t] * f_i:
//   norm   x <- x * w / sqrt(mean(x^2) + eps)              (where a weight is given)
//   turn   (x1, x2)_i <- A (x1 cos a_i - x2 sin a_i, x2 cos a_i + x1 sin a_i)
// over the first rot_dim elements; pair i is elements (i, i + rot_dim / 2) or
// (2i, 2i + 1). Rotated queries go to rows, rotated keys to rows or, with the
// values, to the slot that the row's entry names in the paged pools. All
// arithmetic is in 32 bits with one rounding at the store.
//
// Angles. f_i comes as a 64-bit fraction of a turn, so the angle of any 32-bit
// position, reduced to one turn, is one integer product modulo 2^64: exact but
// for the fraction's own 2^-53 relative rounding (3e-10 rad a million
// positions away), with no 64-bit floating point and no table to read. The top
// 32 bits are split into the nearest quarter turn and a remainder of at most an
// eighth, whose sine and cosine are taken in 32 bits.
//
// Layout. A thread holds two 16-byte vectors of a head, both ends of its pairs
// (half layout) or whole pairs (interleaved), so that a rotation needs no
// exchange and rows may be rotated in place. 8 threads hold a 128-element
// bf16 head; a warp takes 4 heads at a time and goes over the heads of one
// row, so a thread's 8 sines and cosines serve all its heads (few rows: several
// warps share a row). The bytes bound it -- every element is read once and
// written once: 16421 rows of 32 + 8 heads 52.2 us, 6.44 TB/s (54.6 over two sets
// of buffers in turn, of which L2 keeps less); 16384 rows of float32 99.5 us, 6.75
// TB/s -- until the norms come in, whose arithmetic fills 47 % of the issue slots:
// 32768 rows of 32 + 8 + 8 heads 136.8 us, 5.89 TB/s (126 us without norms), 16384
// of float32 128.0 us, 6.29 TB/s. Few rows are bound by the launch and one round
// trip: 64 rows 2.4 us, 2.8 us with the cache write; 2.8 and 3.3 us in float32.
// A ring of rows in shared memory filled by bulk copies, instead of loads held in
// registers, measured 153 us for the 32768 rows and 61 us for 16384 rows without
// norms.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 4;   // warps a block

struct RopeArgs {
    const void *q, *k, *v;          // rows: [T][H][D], row strides in elements
    void *q_out, *k_out;            // k_out: rows, or null with the pools
    void *kpool, *vpool;
    const int32_t* positions;
    const int64_t* slots;
    const void *q_weight, *k_weight;  // [D] or null
    int* err;
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;
    int64_t num_slots;
    int T, Hq, Hk, rot, shift;
    int wpt, gpw;                   // warps a row, head groups a warp
    float eps, amplitude;
    uint64_t turn[PA_ROPE_MAX_PAIRS];
};

// sin and cos of pos * turn (a 2^-64 fraction of a turn a position).
__device__ __forceinline__ float2 sin_cos(int pos, uint64_t turn) {
    const uint32_t ph = static_cast<uint32_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn >> 32);
    const uint32_t quarter = (ph + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(ph - (quarter << 30));  // +- an eighth of a turn
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    const float s1 = quarter & 1 ? c : s, c1 = quarter & 1 ? s : c;
    return make_float2(quarter & 2 ? -s1 : s1, (quarter + 1) & 2 ? -c1 : c1);
}

// A thread's two 16-byte vectors of a head as the two ends of its N pairs, two
// pairs to a 64-bit register for the paired arithmetic: with the half layout
// one vector holds the first ends and the other the second, with the
// interleaved one both hold whole pairs.
template <typename T, bool HALF>
struct Pairs;
template <bool HALF>
struct Pairs<uint16_t, HALF> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 w0, uint4 w1, uint64_t (&x1)[4], uint64_t (&x2)[4]) {
        const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x1[i] = HALF ? f32x2(bf16_lo(u[i]), bf16_hi(u[i])) : f32x2(bf16_lo(u[2 * i]), bf16_lo(u[2 * i + 1]));
            x2[i] = HALF ? f32x2(bf16_lo(u[i + 4]), bf16_hi(u[i + 4]))
                         : f32x2(bf16_hi(u[2 * i]), bf16_hi(u[2 * i + 1]));
        }
    }
    static __device__ __forceinline__ void pack(const uint64_t (&x1)[4], const uint64_t (&x2)[4], uint4& w0, uint4& w1) {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = f32x2_split(x1[i]), b = f32x2_split(x2[i]);
            u[HALF ? i : 2 * i] = HALF ? pack_bf16x2(a.x, a.y) : pack_bf16x2(a.x, b.x);
            u[HALF ? i + 4 : 2 * i + 1] = HALF ? pack_bf16x2(b.x, b.y) : pack_bf16x2(a.y, b.y);
        }
        w0 = make_uint4(u[0], u[1], u[2], u[3]);
        w1 = make_uint4(u[4], u[5], u[6], u[7]);
    }
};
template <bool HALF>
struct Pairs<float, HALF> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 w0, uint4 w1, uint64_t (&x1)[2], uint64_t (&x2)[2]) {
        const float f[8] = {__uint_as_float(w0.x), __uint_as_float(w0.y), __uint_as_float(w0.z),
                            __uint_as_float(w0.w), __uint_as_float(w1.x), __uint_as_float(w1.y),
                            __uint_as_float(w1.z), __uint_as_float(w1.w)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x1[i] = HALF ? f32x2(f[2 * i], f[2 * i + 1]) : f32x2(f[4 * i], f[4 * i + 2]);
            x2[i] = HALF ? f32x2(f[4 + 2 * i], f[5 + 2 * i]) : f32x2(f[4 * i + 1], f[4 * i + 3]);
        }
    }
    static __device__ __forceinline__ void pack(const uint64_t (&x1)[2], const uint64_t (&x2)[2], uint4& w0, uint4& w1) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 a = f32x2_split(x1[i]), b = f32x2_split(x2[i]);
            f[HALF ? 2 * i : 4 * i] = a.x;
            f[HALF ? 2 * i + 1 : 4 * i + 2] = a.y;
            f[HALF ? 4 + 2 * i : 4 * i + 1] = b.x;
            f[HALF ? 5 + 2 * i : 4 * i + 3] = b.y;
        }
        w0 = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        w1 = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
};

// BATCH: groups whose loads are in flight together; BLOCKS: blocks an SM holds at
// least (a bound on registers); WHOLE: a group's heads are all queries or all keys.
template <typename T, int D, bool HALF, bool APPEND, int BATCH, int BLOCKS, bool WHOLE>
__global__ void __launch_bounds__(32 * kRopeWarps, BLOCKS) rope_kernel(const __grid_constant__ RopeArgs a) {
    using P = Pairs<T, HALF>;
    constexpr int N = P::N;           // elements a vector, pairs a thread
    constexpr int TPH = D / (2 * N);  // threads a head
    constexpr int HPW = 32 / TPH;     // heads a warp takes at a time: a group
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int t = a.wpt == 1 ? static_cast<int>(gw) : static_cast<int>(gw / a.wpt);
    if (t >= a.T) return;
    const int g0 = a.wpt == 1 ? 0 : static_cast<int>(gw - static_cast<int64_t>(t) * a.wpt) * a.gpw;
    const int g1 = g0 + a.gpw;  // this warp's groups: of the rotated heads, then of the values
    int64_t slot = 0;
    if constexpr (APPEND) {
        slot = a.slots[t];
        if (slot < 0 || slot >= a.num_slots) {  // -1: a padding row
            if (slot != -1 && lane == 0) atomicOr(a.err, kErrTable);
            return;
        }
    }
    const int pos = a.positions[t];
    const int64_t at = APPEND ? (((slot >> a.shift) * a.Hk << a.shift) + (slot & ((1 << a.shift) - 1))) * D
                              : static_cast<int64_t>(t) * a.ko_stride;
    const int kv_step = APPEND ? D << a.shift : D;  // from a head to the next of the keys' and values' outputs
    const int rotated = (a.Hq + a.Hk + HPW - 1) / HPW;
    // This thread's two vectors of a head, and whether they are rotated.
    const int c = lane % TPH;
    int v0, v1;
    bool r0, r1;
    if constexpr (HALF) {
        const int n2 = a.rot / (2 * N);
        r0 = r1 = c < n2;
        v0 = r0 ? c : 2 * c;       // past the rotated part: 2 n2 + 2 (c - n2)
        v1 = r0 ? n2 + c : 2 * c + 1;
    } else {
        v0 = c;
        v1 = c + TPH;
        r0 = v0 * N < a.rot;
        r1 = v1 * N < a.rot;
    }
    uint64_t sn[N / 2], cs[N / 2];  // sines and cosines of this thread's pairs, two a register
    bool have_angles = false;
    // Groups f .. l - 1 of H heads: kind(h) tells the keys' heads from the queries',
    // src(h) and dst(h) where a head's elements come from and go to.
    auto turn = [&](auto is_key, auto src, auto dst, int H, int f, int l) {
        uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;  // this thread's weights of the kind at hand
        int weight_kind = -1;
        for (int g = f; g < l; g += BATCH) {
            // Every load of the batch before any use.
            uint4 w0[BATCH], w1[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int h = (g + j) * HPW + lane / TPH;
                w0[j] = w1[j] = make_uint4(0, 0, 0, 0);
                if (g + j < l && h < H) {
                    w0[j] = *reinterpret_cast<const uint4*>(src(h) + v0 * N);
                    w1[j] = *reinterpret_cast<const uint4*>(src(h) + v1 * N);
                }
            }
            if (!have_angles) {
                // While they are on their way: each lane takes the sines and
                // cosines of pairs 2 lane and 2 lane + 1, and every thread
                // fetches those of its own pairs from their lanes (16 shuffles
                // in place of 6 more evaluations).
                have_angles = true;
                float2 mine[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mine[e] = make_float2(0.f, 1.f);
                    if (2 * lane + e < a.rot / 2) mine[e] = sin_cos(pos, a.turn[2 * lane + e]);
                    mine[e].x *= a.amplitude;
                    mine[e].y *= a.amplitude;
                }
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const int pair = HALF ? c * N + i : (i < N / 2 ? v0 * (N / 2) + i : v1 * (N / 2) + i - N / 2);
                    const int from = (pair >> 1) & 31;  // pair is even
                    sn[i / 2] = f32x2(__shfl_sync(0xffffffffu, mine[0].x, from), __shfl_sync(0xffffffffu, mine[1].x, from));
                    cs[i / 2] = f32x2(__shfl_sync(0xffffffffu, mine[0].y, from), __shfl_sync(0xffffffffu, mine[1].y, from));
                }
            }
            float ss[BATCH];
            if (a.q_weight || a.k_weight) {  // the shuffles of the batch overlap
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    uint64_t x1[N / 2], x2[N / 2];
                    P::unpack(w0[j], w1[j], x1, x2);
                    uint64_t s1 = f32x2(0.f, 0.f), s2 = s1;
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        s1 = fma_f32x2(x1[i], x1[i], s1);
                        s2 = fma_f32x2(x2[i], x2[i], s2);
                    }
                    const float2 s = f32x2_split(add_f32x2(s1, s2));
                    ss[j] = s.x + s.y;
                }
#pragma unroll
                for (int off = TPH / 2; off > 0; off >>= 1)
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], off);
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int h = (g + j) * HPW + lane / TPH;
                const int key = is_key(h);
                const T* weight = static_cast<const T*>(key ? a.k_weight : a.q_weight);
                uint64_t x1[N / 2], x2[N / 2];
                P::unpack(w0[j], w1[j], x1, x2);
                if (weight) {
                    if (weight_kind != key) {
                        q0 = *reinterpret_cast<const uint4*>(weight + v0 * N);
                        q1 = *reinterpret_cast<const uint4*>(weight + v1 * N);
                        weight_kind = key;
                    }
                    const float r = rsqrtf(ss[j] * (1.f / D) + a.eps);
                    const uint64_t rr = f32x2(r, r);
                    uint64_t y1[N / 2], y2[N / 2];
                    P::unpack(q0, q1, y1, y2);
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
                        const float2 n2 = f32x2_split(z2);
                        x1[i] = fma_f32x2(f32x2(-n2.x, -n2.y), sn[i], mul_f32x2(z1, cs[i]));
                        x2[i] = fma_f32x2(z1, sn[i], mul_f32x2(z2, cs[i]));
                    }
                }
                // A vector that is neither normalised nor rotated keeps its bits.
                uint4 o0, o1;
                P::pack(x1, x2, o0, o1);
                if (weight || r0) w0[j] = o0;
                if (weight || r1) w1[j] = o1;
                if (g + j < l && h < H) {
                    *reinterpret_cast<uint4*>(dst(h) + v0 * N) = w0[j];
                    *reinterpret_cast<uint4*>(dst(h) + v1 * N) = w1[j];
                }
            }
        }
    };
    {
        const T* const src_q = static_cast<const T*>(a.q) + static_cast<int64_t>(t) * a.q_stride;
        const T* const src_k = static_cast<const T*>(a.k) + static_cast<int64_t>(t) * a.k_stride;
        T* const dst_q = static_cast<T*>(a.q_out) + static_cast<int64_t>(t) * a.qo_stride;
        T* const dst_k = static_cast<T*>(APPEND ? a.kpool : a.k_out) + at;
        if constexpr (WHOLE) {
            // Whole groups of queries, then of keys: nothing to select per head.
            const int nq = a.Hq / HPW;
            turn([](int) { return 0; }, [&](int h) { return src_q + h * D; }, [&](int h) { return dst_q + h * D; },
                 a.Hq, min(g0, nq), min(g1, nq));
            turn([](int) { return 1; }, [&](int h) { return src_k + h * D; },
                 [&](int h) { return dst_k + static_cast<int64_t>(h) * kv_step; }, a.Hk, max(g0 - nq, 0),
                 min(g1, rotated) - nq);
        } else {
            turn([&](int h) { return h < a.Hq ? 0 : 1; },
                 [&](int h) { return h < a.Hq ? src_q + h * D : src_k + (h - a.Hq) * D; },
                 [&](int h) { return h < a.Hq ? dst_q + h * D : dst_k + static_cast<int64_t>(h - a.Hq) * kv_step; },
                 a.Hq + a.Hk, g0, min(g1, rotated));
        }
    }
    if constexpr (APPEND) {
        // The values' groups: copied, vector by vector.
        constexpr int VPH = D / N;  // vectors a head
        const T* const src = static_cast<const T*>(a.v) + static_cast<int64_t>(t) * a.v_stride;
        T* const dst = static_cast<T*>(a.vpool) + at;
        const int end = min(g1 - rotated, (a.Hk + HPW - 1) / HPW) * HPW * VPH;
        for (int i = max(g0 - rotated, 0) * HPW * VPH + lane; i < end; i += 32 * 4) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + 32 * j < min(end, a.Hk * VPH)) w[j] = *reinterpret_cast<const uint4*>(src + (i + 32 * j) * N);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int h = (i + 32 * j) / VPH, e = (i + 32 * j) % VPH;
                if (i + 32 * j < min(end, a.Hk * VPH))
                    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(h) * kv_step + e * N) = w[j];
            }
        }
    }
}

using RopeFn = void (*)(RopeArgs);

template <bool APPEND, int BATCH, int BLOCKS, bool WHOLE>
RopeFn rope_select(int D, bool bf16, bool half) {
    if (bf16 && D == 128)
        return half ? rope_kernel<uint16_t, 128, true, APPEND, BATCH, BLOCKS, WHOLE>
                    : rope_kernel<uint16_t, 128, false, APPEND, BATCH, BLOCKS, WHOLE>;
    if (bf16)
        return half ? rope_kernel<uint16_t, 64, true, APPEND, BATCH, BLOCKS, WHOLE>
                    : rope_kernel<uint16_t, 64, false, APPEND, BATCH, BLOCKS, WHOLE>;
    if (D == 128)
        return half ? rope_kernel<float, 128, true, APPEND, BATCH, BLOCKS, WHOLE>
                    : rope_kernel<float, 128, false, APPEND, BATCH, BLOCKS, WHOLE>;
    return half ? rope_kernel<float, 64, true, APPEND, BATCH, BLOCKS, WHOLE>
                : rope_kernel<float, 64, false, APPEND, BATCH, BLOCKS, WHOLE>;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A row stride (elements): whole 16-byte vectors, at least a row.
bool stride_ok(int64_t stride, int H, int D, int elem) {
    return stride >= static_cast<int64_t>(H) * D && stride * elem % 16 == 0;
}

// The arguments that both calls share.
pa_status rope_args(RopeArgs* a, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                    const int32_t* positions, int T, int Hq, int Hk, int D, pa_dtype dtype,
                    const void* q_weight, const void* k_weight, float eps, const pa_rope* rope,
                    void* q_out, int64_t qo_stride) {
    if (!q || !k || !positions || !q_out) return PA_ERR_NULL;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_DTYPE;
    const int elem = dtype == PA_F32 ? 4 : 2;
    if (T < 0 || Hq < 1 || Hk < 1 || Hq > 65536 || Hk > 65536 || (D != 64 && D != 128) ||
        !stride_ok(q_stride, Hq, D, elem) || !stride_ok(k_stride, Hk, D, elem) ||
        !stride_ok(qo_stride, Hq, D, elem) || !(eps >= 0.f) || !std::isfinite(eps))
        return PA_ERR_SHAPE;
    if (rope && (rope->rot_dim < 16 || rope->rot_dim > D || rope->rot_dim % 16 != 0 ||
                 (rope->layout != PA_ROPE_HALF && rope->layout != PA_ROPE_INTERLEAVED) ||
                 !std::isfinite(rope->amplitude)))
        return PA_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || (q_weight && !aligned16(q_weight)) ||
        (k_weight && !aligned16(k_weight)) || (reinterpret_cast<uintptr_t>(positions) & 3u))
        return PA_ERR_ALIGN;
    a->q = q;
    a->k = k;
    a->q_out = q_out;
    a->positions = positions;
    a->q_weight = q_weight;
    a->k_weight = k_weight;
    a->q_stride = q_stride;
    a->k_stride = k_stride;
    a->qo_stride = qo_stride;
    a->T = T;
    a->Hq = Hq;
    a->Hk = Hk;
    a->eps = eps;
    if (rope) {
        a->rot = rope->rot_dim;
        a->amplitude = rope->amplitude;
        for (int i = 0; i < rope->rot_dim / 2; ++i) a->turn[i] = rope->turn[i];
    }
    return PA_OK;
}

template <bool APPEND>
pa_status rope_launch(RopeArgs* a, int D, bool bf16, bool half, cudaStream_t stream) {
    if (a->T == 0) return PA_OK;
    const int hpw = 32 / (D / (32 / (bf16 ? 2 : 4)));
    const int groups = (a->Hq + a->Hk + hpw - 1) / hpw + (APPEND ? (a->Hk + hpw - 1) / hpw : 0);
    // One warp a row, all its heads, once the rows alone fill the SMs; more
    // warps a row, each with fewer heads, before that.
    const int64_t fill = static_cast<int64_t>(kSms) * 16;
    a->wpt = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(groups, (fill + a->T - 1) / a->T)));
    a->gpw = (groups + a->wpt - 1) / a->wpt;
    a->wpt = (groups + a->gpw - 1) / a->gpw;
    // Queries and keys in loops of their own where both fill whole groups and
    // the queries alone a few of them (32768 rows of 32 + 8 + 8 heads with norms
    // 135 against 146 us); one loop over both otherwise (32768 rows of 4 + 4
    // heads 35 against 42 us), so that few heads still share a batch of loads.
    // Loads in flight: four groups, or two beside the norm's and the pools'
    // registers (16421 rows of 32 + 8 heads 51.9 us with four and 52.9 with
    // two; the 32768 rows above 135.2 us with two and 136.6 with four).
    const bool whole = a->Hq % hpw == 0 && a->Hk % hpw == 0 && a->Hq >= 4 * hpw;
    const RopeFn fn = a->gpw == 1 ? rope_select<APPEND, 1, 1, false>(D, bf16, half)
                      : whole     ? rope_select<APPEND, APPEND ? 2 : 4, 5, true>(D, bf16, half)
                                  : rope_select<APPEND, 2, 5, false>(D, bf16, half);
    const int64_t blocks = (static_cast<int64_t>(a->T) * a->wpt + kRopeWarps - 1) / kRopeWarps;
    if (blocks > INT32_MAX) return PA_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(32 * kRopeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, *a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_rope_inv_freq(int rot_dim, double base, int scaling, double factor, double orig_len,
                           double low_turns, double high_turns, double* inv_freq, float* amplitude) {
    if (!inv_freq || !amplitude) return PA_ERR_NULL;
    if (rot_dim < 16 || rot_dim > 2 * PA_ROPE_MAX_PAIRS || rot_dim % 16 != 0 || !(base > 1.0) ||
        !std::isfinite(base) || scaling < PA_ROPE_NONE || scaling > PA_ROPE_YARN)
        return PA_ERR_SHAPE;
    if (scaling != PA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return PA_ERR_SHAPE;
    const bool ramp = scaling == PA_ROPE_PARTS || scaling == PA_ROPE_YARN;
    if (ramp && (!(orig_len >= 1.0) || !std::isfinite(orig_len) || !(low_turns > 0.0) ||
                 !(high_turns > low_turns) || !std::isfinite(high_turns)))
        return PA_ERR_SHAPE;
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const int n = rot_dim / 2;
    // The pair index at which a pair makes the given number of turns over orig_len.
    auto index_at = [&](double turns) {
        return rot_dim * std::log(orig_len / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    double first = 0.0, last = 0.0;
    if (scaling == PA_ROPE_YARN) {
        first = std::max(std::floor(index_at(high_turns)), 0.0);
        last = std::min(std::ceil(index_at(low_turns)), static_cast<double>(rot_dim - 1));
        if (last <= first) last = first + 0.001;
    }
    for (int i = 0; i < n; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        double keep = 1.0;  // share of the unscaled frequency
        if (scaling == PA_ROPE_LINEAR) keep = 0.0;
        if (scaling == PA_ROPE_PARTS)
            keep = (orig_len * f / kTwoPi - low_turns) / (high_turns - low_turns);
        if (scaling == PA_ROPE_YARN) keep = 1.0 - (i - first) / (last - first);
        keep = std::min(1.0, std::max(0.0, keep));
        inv_freq[i] = scaling == PA_ROPE_NONE ? f : keep * f + (1.0 - keep) * f / factor;
    }
    *amplitude = scaling == PA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
    return PA_OK;
}

pa_status pa_rope_init(pa_rope* rope, int rot_dim, int layout, const double* inv_freq,
                       float amplitude) {
    if (!rope || !inv_freq) return PA_ERR_NULL;
    if (rot_dim < 16 || rot_dim > 2 * PA_ROPE_MAX_PAIRS || rot_dim % 16 != 0 ||
        (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED) || !std::isfinite(amplitude))
        return PA_ERR_SHAPE;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i])) return PA_ERR_SHAPE;
    *rope = pa_rope{};
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    rope->amplitude = amplitude;
    for (int i = 0; i < rot_dim / 2; ++i) {
        // Whole turns drop out of the angle at every integer position.
        const double turns = inv_freq[i] / 6.283185307179586476925286766559;
        const double part = turns - std::floor(turns);  // [0, 1], 1 only by rounding
        rope->turn[i] = part < 1.0 ? static_cast<uint64_t>(std::ldexp(part, 64)) : 0;
    }
    return PA_OK;
}

pa_status pa_qk_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const int32_t* positions, int num_rows, int Hq, int Hk, int D, pa_dtype dtype,
                     const void* q_weight, const void* k_weight, float eps, const pa_rope* rope,
                     void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                     struct CUstream_st* stream) {
    pa::RopeArgs a{};
    if (!k_out) return PA_ERR_NULL;
    const pa_status st = pa::rope_args(&a, q, q_stride, k, k_stride, positions, num_rows, Hq, Hk, D,
                                       dtype, q_weight, k_weight, eps, rope, q_out, q_out_stride);
    if (st != PA_OK) return st;
    const int elem = dtype == PA_F32 ? 4 : 2;
    if (!pa::stride_ok(k_out_stride, Hk, D, elem)) return PA_ERR_SHAPE;
    if (!pa::aligned16(k_out)) return PA_ERR_ALIGN;
    a.k_out = k_out;
    a.ko_stride = k_out_stride;
    return pa::rope_launch<false>(&a, D, dtype == PA_BF16, !rope || rope->layout == PA_ROPE_HALF,
                                  reinterpret_cast<cudaStream_t>(stream));
}

pa_status pa_qk_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* v, int64_t v_stride, const int32_t* positions,
                            const int64_t* slots, int num_rows, int Hq, int Hkv, int D,
                            pa_dtype dtype, const void* q_weight, const void* k_weight, float eps,
                            const pa_rope* rope, void* q_out, int64_t q_out_stride, void* k_pool,
                            void* v_pool, int block_size, int num_blocks, int* device_error,
                            struct CUstream_st* stream) {
    if (!v || !slots || !k_pool || !v_pool) return PA_ERR_NULL;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    pa::RopeArgs a{};
    const pa_status st = pa::rope_args(&a, q, q_stride, k, k_stride, positions, num_rows, Hq, Hkv, D,
                                       dtype, q_weight, k_weight, eps, rope, q_out, q_out_stride);
    if (st != PA_OK) return st;
    const int elem = dtype == PA_F32 ? 4 : 2;
    if (!pa::stride_ok(v_stride, Hkv, D, elem) || num_blocks < 1) return PA_ERR_SHAPE;
    if (!pa::aligned16(v) || !pa::aligned16(k_pool) || !pa::aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u) || (reinterpret_cast<uintptr_t>(device_error) & 3u))
        return PA_ERR_ALIGN;
    a.v = v;
    a.v_stride = v_stride;
    a.slots = slots;
    a.kpool = k_pool;
    a.vpool = v_pool;
    a.shift = block_size == 16 ? 4 : 5;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.err = device_error;
    if (num_rows > 0 && !a.err && pa::append_error_address(&a.err) != cudaSuccess) return PA_ERR_CUDA;
    return pa::rope_launch<true>(&a, D, dtype == PA_BF16, !rope || rope->layout == PA_ROPE_HALF,
                                 reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
