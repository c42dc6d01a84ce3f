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
// row, so a thread's 8 sines and cosines serve all its heads. The bytes bound
// it: every element is read once and written once.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kRopeWarps = 4;  // warps a block

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

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 w, float* x) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(u[i]);
            x[2 * i + 1] = bf16_hi(u[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 w, float* x) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <typename T, int D, bool HALF, bool APPEND>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int N = Vec<T>::N;      // elements a vector
    constexpr int TPH = D / (2 * N);  // threads a head
    constexpr int HPW = 32 / TPH;     // heads a warp takes at a time
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t gw = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
    const int t = static_cast<int>(gw / a.wpt);
    if (t >= a.T) return;
    const int g0 = static_cast<int>(gw - static_cast<int64_t>(t) * a.wpt) * a.gpw;
    const int heads = a.Hq + (APPEND ? 2 : 1) * a.Hk;
    const int groups = (heads + HPW - 1) / HPW;
    const int g1 = min(g0 + a.gpw, groups);
    int64_t slot = 0;
    if constexpr (APPEND) {
        slot = a.slots[t];
        if (slot < 0 || slot >= a.num_slots) {  // -1: a padding row
            if (slot != -1 && lane == 0) atomicOr(a.err, kErrTable);
            return;
        }
    }
    const int pos = a.positions[t];
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
    struct Group {       // this thread's part of a group of heads
        uint4 w0, w1;
        T* dst;
        int kind;        // 0: q, 1: k, 2: v, 3: no head
    };
    auto load = [&](int g) {
        const int head = g * HPW + lane / TPH;
        Group r;
        r.kind = head < a.Hq ? 0 : head < a.Hq + a.Hk ? 1 : head < heads ? 2 : 3;
        const int h = head - (r.kind == 0 ? 0 : r.kind == 1 ? a.Hq : a.Hq + a.Hk);
        r.w0 = r.w1 = make_uint4(0, 0, 0, 0);
        r.dst = nullptr;
        if (r.kind < 3) {
            const T* src = static_cast<const T*>(r.kind == 0 ? a.q : r.kind == 1 ? a.k : a.v) +
                           static_cast<int64_t>(t) * (r.kind == 0 ? a.q_stride : r.kind == 1 ? a.k_stride : a.v_stride) +
                           h * D;
            r.w0 = *reinterpret_cast<const uint4*>(src + v0 * N);
            r.w1 = *reinterpret_cast<const uint4*>(src + v1 * N);
            if (r.kind == 0) {
                r.dst = static_cast<T*>(a.q_out) + static_cast<int64_t>(t) * a.qo_stride + h * D;
            } else if constexpr (APPEND) {
                r.dst = static_cast<T*>(r.kind == 1 ? a.kpool : a.vpool) +
                        ((((slot >> a.shift) * a.Hk + h) << a.shift) + (slot & ((1 << a.shift) - 1))) * D;
            } else {
                r.dst = static_cast<T*>(a.k_out) + static_cast<int64_t>(t) * a.ko_stride + h * D;
            }
        }
        return r;
    };
    Group next = load(g0);
    float2 sc[N];  // sin, cos: pair by pair
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pair = HALF ? c * N + i : (i < N / 2 ? v0 * (N / 2) + i : v1 * (N / 2) + i - N / 2);
        const bool on = HALF ? r0 : (i < N / 2 ? r0 : r1);
        sc[i] = make_float2(0.f, 1.f);
        if (on) {
            sc[i] = sin_cos(pos, a.turn[pair]);
            sc[i].x *= a.amplitude;
            sc[i].y *= a.amplitude;
        }
    }
    // The vectors of the next group are on their way while one is worked on.
    for (int g = g0; g < g1; ++g) {
        const Group now = next;
        if (g + 1 < g1) next = load(g + 1);
        const bool is_q = now.kind == 0, turn = now.kind <= 1;
        const T* weight = static_cast<const T*>(is_q ? a.q_weight : now.kind == 1 ? a.k_weight : nullptr);
        float x[2 * N];
        Vec<T>::unpack(now.w0, x);
        Vec<T>::unpack(now.w1, x + N);
        const bool norm = weight != nullptr;
        if (__any_sync(0xffffffffu, norm)) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int off = TPH / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            if (norm) {
                const float r = rsqrtf(ss * (1.f / D) + a.eps);
                float wt[2 * N];
                Vec<T>::unpack(*reinterpret_cast<const uint4*>(weight + v0 * N), wt);
                Vec<T>::unpack(*reinterpret_cast<const uint4*>(weight + v1 * N), wt + N);
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) x[i] *= r * wt[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e1 = HALF ? i : 2 * i, e2 = HALF ? i + N : 2 * i + 1;
            const bool rot = turn && (HALF ? r0 : (i < N / 2 ? r0 : r1));
            const float x1 = x[e1], x2 = x[e2];
            if (rot) {
                x[e1] = x1 * sc[i].y - x2 * sc[i].x;
                x[e2] = x2 * sc[i].y + x1 * sc[i].x;
            }
        }
        // A vector that is neither normalised nor rotated keeps its bits.
        const uint4 w0 = norm || (turn && r0) ? Vec<T>::pack(x) : now.w0;
        const uint4 w1 = norm || (turn && r1) ? Vec<T>::pack(x + N) : now.w1;
        if (now.kind < 3) {
            *reinterpret_cast<uint4*>(now.dst + v0 * N) = w0;
            *reinterpret_cast<uint4*>(now.dst + v1 * N) = w1;
        }
    }
}

using RopeFn = void (*)(RopeArgs);

template <bool APPEND>
RopeFn rope_select(int D, bool bf16, bool half) {
    if (bf16) {
        if (D == 128) return half ? rope_kernel<uint16_t, 128, true, APPEND> : rope_kernel<uint16_t, 128, false, APPEND>;
        return half ? rope_kernel<uint16_t, 64, true, APPEND> : rope_kernel<uint16_t, 64, false, APPEND>;
    }
    if (D == 128) return half ? rope_kernel<float, 128, true, APPEND> : rope_kernel<float, 128, false, APPEND>;
    return half ? rope_kernel<float, 64, true, APPEND> : rope_kernel<float, 64, false, APPEND>;
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
        (k_weight && !aligned16(k_weight)))
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

pa_status rope_launch(RopeArgs* a, RopeFn fn, int heads, int D, int elem, cudaStream_t stream) {
    if (a->T == 0) return PA_OK;
    const int hpw = 32 / (D / (32 / elem));
    const int groups = (heads + hpw - 1) / hpw;
    // One warp a row, all its heads, once the rows alone fill the SMs; more
    // warps a row, each with fewer heads, before that.
    const int64_t fill = 152LL * 32;
    a->wpt = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(groups, (fill + a->T - 1) / a->T)));
    a->gpw = (groups + a->wpt - 1) / a->wpt;
    a->wpt = (groups + a->gpw - 1) / a->gpw;
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
    return pa::rope_launch(&a, pa::rope_select<false>(D, dtype == PA_BF16,
                                                      !rope || rope->layout == PA_ROPE_HALF),
                           Hq + Hk, D, elem, reinterpret_cast<cudaStream_t>(stream));
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
    if (!pa::aligned16(v) || !pa::aligned16(k_pool) || !pa::aligned16(v_pool)) return PA_ERR_ALIGN;
    a.v = v;
    a.v_stride = v_stride;
    a.slots = slots;
    a.kpool = k_pool;
    a.vpool = v_pool;
    a.shift = block_size == 16 ? 4 : 5;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.err = device_error;
    if (num_rows > 0 && !a.err && pa::append_error_address(&a.err) != cudaSuccess) return PA_ERR_CUDA;
    return pa::rope_launch(&a, pa::rope_select<true>(D, dtype == PA_BF16,
                                                     !rope || rope->layout == PA_ROPE_HALF),
                           Hq + 2 * Hkv, D, elem, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
