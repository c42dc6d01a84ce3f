// Paged decode attention with a sliding window and sinks (pa_decode_window):
// one new query per sequence, over the tokens t >= L - W and t < S.
//
// With a window every (sequence, kv unit) segment whose context is past it costs
// the same, min(L, W + S) tokens, whatever the context's length. So the work is not
// cut out of one long page stream (pa_split.cuh) but laid out by segment: a segment's
// visible pages (WindowView) are divided among the warps of one block, or of a
// cluster of up to 8 blocks where there are few segments, and the warps'
// partial results (m, l, acc) are merged on the chip -- in shared memory, then
// across the cluster through distributed shared memory -- with m = max m_i,
// l = sum l_i 2^(m_i - m), o = sum acc_i 2^(m_i - m) / l ("39 · PagedAttention"
// §3). No partial goes to memory and no second kernel follows.
//
// Each warp takes every W-th 32-token chunk of its block's range: lane 0 moves
// the chunk's pages into the warp's stage with tiled bulk tensor copies (128-byte
// swizzle) and the warp runs the split decode's tensor-core tile on it (scores
// S^T = K Q^T, probabilities as a bf16 pair hi + lo, O^T += V^T P^T, running
// maximum in the log2 domain; pa_split.cuh's MmaState). Twelve such warps fill an
// SM's shared memory at D = 128, in one, two or four blocks; at D = 64, with half
// the bytes a warp, registers allow 18 (15 above 8 heads a kv head). DRAM bounds it
// for many segments, less the last blocks' uneven end: 64 sequences of 8 kv heads,
// W = 1024, 45.4 us, 5.8 TB/s; 128 of 32, W = 4096, 1143 us, 7.5 TB/s. For few, the
// latency of a chunk's copies and of the merge bounds it, and the SMs that a cluster
// a segment leaves idle: one sequence of 8 kv heads, W = 8191, 64 blocks, 13.8 us,
// 2.5 TB/s (11.5 with the pages in L2). Blocks and warps are cut for the host's
// bound on the visible tokens, so contexts of many lengths below the window take up
// to 3 times their bytes' time: 32 sequences of 16 to 8192 tokens, 8 kv heads, W =
// 4096, 47 us for 119 MB.
#include "pa_split.cuh"

#include <algorithm>

#include "pa.h"

namespace pa {
namespace {

constexpr int kWarpsPerSm = 12;

struct WindowDecodeArgs {
    const uint16_t* q;         // [B][Hq][D] bf16 bits
    const int32_t* tables;     // [B][max_blocks]
    const int32_t* seq_lens;   // [B]
    void* out;                 // [B][Hq][D], bf16 or f32
    int* err;
    int B, Hq, Hkv, g;         // g = Hq / Hkv
    int GS, nslices, U;        // q heads per slice, slices per kv head, U = Hkv * nslices
    int max_blocks, num_blocks, max_seq_len;
    int window, sinks;
    int cluster;               // blocks per segment
    float scale_log2;
    int out_bf16, probe_wait;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of the cluster: what was written to shared memory before is
// visible to all after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same shared-memory address in block `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// A partial result in shared memory: acc [GS][D], then (m, l) [GS]. m = -inf: no
// token; m = NaN: a bad table entry or a copy that never arrived.
__host__ __device__ constexpr uint32_t part_bytes(int GS, int D) { return (GS * D * 4u + GS * 8u + 15u) & ~15u; }

// Folds n partials of unit (head, 4 elements) into (m, l, acc), m and l from
// load_ml(i) and the elements from load_acc(i).
template <typename Ml, typename Acc>
__device__ __forceinline__ void fold(int n, Ml load_ml, Acc load_acc, float& m, float& l, float4& acc) {
    m = -INFINITY;
    bool poison = false;
    for (int i = 0; i < n; ++i) {
        const float mi = load_ml(i).x;
        poison |= mi != mi;
        m = fmaxf(m, mi);  // fmaxf passes over NaN
    }
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (poison) {
        m = __int_as_float(0x7fc00000);
        return;
    }
    if (m == -INFINITY) return;
    for (int i = 0; i < n; ++i) {
        const float2 ml = load_ml(i);
        const float f = fast_exp2(ml.x - m);  // 0 for a partial without a token
        const float4 v = load_acc(i);
        l = fmaf(ml.y, f, l);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
    }
}

template <int D, int BS, int NT>
__global__ void __launch_bounds__(32 * kWarpsPerSm, 1)
    window_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const WindowDecodeArgs a) {
    using State = split::MmaState<D, kChunkTokens, NT, NT == 2>;
    constexpr int CT = kChunkTokens;
    constexpr int CP = CT / BS;                       // pages per chunk
    constexpr uint32_t kStage = 2u * CT * D * 2u;     // K and V of a chunk
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, W = blockDim.x >> 5;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    // Stages; query rows, and in their place at the end the block's partial
    // (read by the cluster); barriers.
    const uint32_t off_part = W * kStage, off_q = off_part;
    const uint32_t off_bar = off_part + part_bytes(a.GS, D);
    const uint32_t stg = base + warp * kStage, bar = base + off_bar + 8 * warp;
    const uint32_t probe_bar = base + off_bar + 8 * W;
    if (tid == 0) {
        for (int w = 0; w <= W; ++w) mbar_init(base + off_bar + 8 * w, 1);  // the last: nothing completes it
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    const int seg = blockIdx.x / a.cluster;
    const int rank = a.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int b = seg / a.U, u = seg - b * a.U;
    const int kvh = u / a.nslices, slice = u - kvh * a.nslices;
    const int nh = min(a.GS, a.g - slice * a.GS);
    const size_t row0 = static_cast<size_t>(b) * a.Hq + kvh * a.g + slice * a.GS;  // first output row
    griddep_wait();
    griddep_launch_dependents();
    const int L = a.seq_lens[b];
    if (L < 1 || L > min(a.max_seq_len, a.max_blocks * BS)) {  // the whole cluster leaves
        if (rank == 0) {
            if (tid == 0) atomicOr(a.err, kErrSeqLen);
            for (int i = tid; i < nh * D; i += blockDim.x) {
                if (a.out_bf16) static_cast<uint16_t*>(a.out)[row0 * D + i] = 0;
                else static_cast<float*>(a.out)[row0 * D + i] = 0.f;
            }
        }
        return;
    }
    const WindowView view = window_view(L - 1, L - 1, a.window, a.sinks, BS);
    const int nb = (view.len + BS - 1) / BS, nch = (nb + CP - 1) / CP;
    const int per = (nch + a.cluster - 1) / a.cluster;
    const int c_end = min(nch, (rank + 1) * per);
    const int32_t* const table = a.tables + static_cast<size_t>(b) * a.max_blocks;
    const int sink_pages = (a.sinks + BS - 1) / BS;
    // Lane j: the block of page j of chunk c (-1 past the end).
    auto entries = [&](int c) {
        const int p = c * CP + lane;
        return lane < CP && p < nb ? __ldg(table + (p < sink_pages ? p : p + view.skip)) : -1;
    };
    int c = rank * per + warp;
    int phys = c < c_end ? entries(c) : -1;
    for (int i = tid; i < nh * (D / 8); i += blockDim.x) {
        const int h = i / (D / 8), e = i - h * (D / 8);
        *reinterpret_cast<uint4*>(gbase + off_q + h * State::QP + e * 16) =
            *reinterpret_cast<const uint4*>(a.q + (row0 + h) * D + e * 8);
    }
    __syncthreads();

    bool poison = false;
    const uint32_t one = elect_one();
    // Copies the chunk's pages into the warp's stage; false if one is outside the pool.
    auto issue = [&](int chunk, int page) {
        const int n = min(CP, nb - chunk * CP);
        const bool bad = __any_sync(0xffffffffu, lane < n && (page < 0 || page >= a.num_blocks));
        if (bad) {
            if (lane == 0) atomicOr(a.err, kErrTable);
            return false;
        }
        if (one) mbar_arrive_expect_tx(bar, n * (2u * BS * D * 2u));
        __syncwarp();
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const int r = __shfl_sync(0xffffffffu, page, j) * a.Hkv + kvh;
            const uint32_t on = j < n ? one : 0u;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint32_t off = h * (CT * 128) + j * (BS * 128);
                tma_load_3d_if(on, stg + off, &kmap, h * 64, 0, r, bar);
                tma_load_3d_if(on, stg + CT * D * 2 + off, &vmap, h * 64, 0, r, bar);
            }
        }
        return true;
    };
    State st;
    const uint32_t qst = base + off_q;
    bool loaded = c < c_end && issue(c, phys);
    poison = c < c_end && !loaded;
    st.start(qst, nh, lane);
    uint32_t phase = 0;
    bool first = true;
    while (loaded) {
        const int next = c + W;
        const int next_phys = next < c_end ? entries(next) : -1;
        const bool ready = a.probe_wait && first ? mbar_wait_bounded(probe_bar, 0, kProbeLimitNs)
                                                 : mbar_wait_bounded(bar, phase, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, ready)) {
            // Give up: report, wait (bounded) for the copies in flight. The
            // block and its cluster still meet at their barriers below.
            if (lane == 0) atomicOr(a.err, kErrTimeout);
            mbar_wait_bounded(bar, phase, kWaitLimitNs);
            poison = true;
            break;
        }
        first = false;
        phase ^= 1u;
        const int v0 = c * CT;
        const int nv = min(min(CP, nb - c * CP) * BS, view.len - v0);
        const int h0 = max(0, min(CT, a.sinks - v0)), h1 = max(0, min(CT, view.lo - v0));
        st.template page<false, true>(stg, stg + CT * D * 2, nv, a.scale_log2, lane, 0, 0, 1, qst, nh, h0, h1);
        __syncwarp();
        c = next;
        loaded = false;
        if (c < c_end) {
            fence_proxy_async_smem();
            loaded = issue(c, next_phys);
            poison = !loaded;
        }
    }

    // This warp's partial into its own stage (its copies are all done).
    {
        float* acc = reinterpret_cast<float*>(gbase + warp * kStage);
        float* ml = acc + a.GS * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = st.l[nt][j];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int head = nt * 8 + 2 * (lane & 3) + j, dr = lane >> 2;
                if (head >= nh) continue;
#pragma unroll
                for (int mt = 0; mt < State::KS; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) acc[head * D + mt * 16 + dr + 8 * r] = st.o[mt][nt][2 * r + j];
                if (dr == 0) {
                    ml[2 * head] = poison ? __int_as_float(0x7fc00000) : st.m[nt][j];
                    ml[2 * head + 1] = l;
                }
            }
        }
    }
    __syncthreads();
    auto store = [&](int head, int d, float m, float l, float4 v) {
        // The marker m = NaN (not NaN data: maxima pass over it) zeroes the row;
        // sums that are NaN because a visible key or value is stay so.
        const float inv = m != m ? 0.f : 1.f / l;
        const size_t o = (row0 + head) * D + d;
        if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) =
                make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    };
    const int units = nh * (D / 4);
    for (int i = tid; i < units; i += blockDim.x) {
        const int head = i / (D / 4), d = (i - head * (D / 4)) * 4;
        float m, l;
        float4 v;
        fold(W, [&](int w) { return *reinterpret_cast<const float2*>(gbase + w * kStage + a.GS * D * 4 + head * 8); },
             [&](int w) { return *reinterpret_cast<const float4*>(gbase + w * kStage + (head * D + d) * 4); }, m, l, v);
        if (a.cluster == 1) {
            store(head, d, m, l, v);
        } else {
            float* part = reinterpret_cast<float*>(gbase + off_part);
            *reinterpret_cast<float4*>(part + head * D + d) = v;
            if (d == 0) *reinterpret_cast<float2*>(part + a.GS * D + 2 * head) = make_float2(m, l);
        }
    }
    if (a.cluster == 1) return;
    // Across the cluster: each block folds its share of the units.
    cluster_sync();
    const uint32_t part = base + off_part;
    for (int i = rank * blockDim.x + tid; i < units; i += a.cluster * blockDim.x) {
        const int head = i / (D / 4), d = (i - head * (D / 4)) * 4;
        float m, l;
        float4 v;
        fold(a.cluster, [&](int r) { return ld_cluster_f2(map_rank(part + (a.GS * D + 2 * head) * 4, r)); },
             [&](int r) { return ld_cluster_f4(map_rank(part + (head * D + d) * 4, r)); }, m, l, v);
        store(head, d, m, l, v);
    }
    cluster_sync();  // no block leaves while another reads its partial
}

using WindowDecodeFn = void (*)(CUtensorMap, CUtensorMap, WindowDecodeArgs);

WindowDecodeFn select_window_decode(int D, int BS, int NT) {
    if (D == 128 && BS == 16) return NT == 1 ? window_decode_kernel<128, 16, 1> : window_decode_kernel<128, 16, 2>;
    if (D == 128) return NT == 1 ? window_decode_kernel<128, 32, 1> : window_decode_kernel<128, 32, 2>;
    if (BS == 16) return NT == 1 ? window_decode_kernel<64, 16, 1> : window_decode_kernel<64, 16, 2>;
    return NT == 1 ? window_decode_kernel<64, 32, 1> : window_decode_kernel<64, 32, 2>;
}

void cluster_launch(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int cluster, int threads, size_t smem) {
    cfg->blockDim = dim3(threads);
    cfg->dynamicSmemBytes = smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

size_t smem_bytes(int W, int GS, int D) {
    return 1024 + static_cast<size_t>(W) * 2 * kChunkTokens * D * 2 + part_bytes(GS, D) + 8 * (W + 1);
}

}  // namespace

// Blocks per SM and per segment: the fewest rounds of chunks, a round being one
// chunk for each of the warps at work, over all waves of blocks (and half a
// round for a merge in the block, one for a merge in the cluster). Measured, us
// (block 16, D = 128): 512 segments of 1028 tokens 44.5 with four blocks an SM
// against 47.3 with two and 54.6 with one; 8 segments of 8255 tokens, blocks of
// 12 warps, 12.1 in clusters of 8 against 16.2 of 4 and 23.8 of 2.
cudaError_t window_decode_shape(int64_t segs, int GS, int D, int block_size, int vis_len, int num_sms,
                                std::vector<WindowRoom>* rooms, WindowDecodeShape* out) {
    const int NT = (GS + 7) / 8;
    const WindowRoom* room = nullptr;
    for (const WindowRoom& r : *rooms)
        if (r.D == D && r.BS == block_size && r.GS == GS) room = &r;
    if (!room) {
        // Clusters the device holds at a time; they depend on how its SMs are
        // grouped (152, 144 and 120 blocks of clusters of 2, 4 and 8 at one
        // block per SM on the measured chip).
        WindowRoom r{D, block_size, GS, {}};
        auto fn = select_window_decode(D, block_size, NT);
        // For this call and the later ones of the plan, whatever their shape.
        cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmemLimit));
        if (e != cudaSuccess) return e;
        for (int i = 0; i < 3; ++i) {
            for (int j = 0; j < 4; ++j) {
                const int W = kWarpsPerSm >> i;
                const size_t smem = smem_bytes(W, GS, D);
                if (j == 0) {
                    int n = 0;
                    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(fn), 32 * W, smem);
                    r.room[i][j] = n * num_sms;
                } else {
                    cudaLaunchConfig_t cfg = {};
                    cudaLaunchAttribute attr[1];
                    cluster_launch(&cfg, attr, 1 << j, 32 * W, smem);
                    cfg.gridDim = dim3(1u << j);
                    e = cudaOccupancyMaxActiveClusters(&r.room[i][j], reinterpret_cast<const void*>(fn), &cfg);
                }
                if (e != cudaSuccess) return e;
            }
        }
        rooms->push_back(r);
        room = &rooms->back();
    }
    const int64_t chunks = (static_cast<int64_t>(vis_len) + kChunkTokens - 1) / kChunkTokens + 1;
    double best = 1e300;
    *out = WindowDecodeShape{};
    for (int i = 2; i >= 0; --i) {
        for (int j = 0; j < 4; ++j) {
            if (room->room[i][j] < 1) continue;
            const int64_t warps = static_cast<int64_t>(kWarpsPerSm >> i) << j;
            const int64_t waves = (segs + room->room[i][j] - 1) / room->room[i][j];
            const int64_t rounds = (chunks + warps - 1) / warps;
            const double cost = static_cast<double>(waves) * (static_cast<double>(rounds) + (j ? 1.0 : 0.5));
            if (cost < best) {
                best = cost;
                *out = WindowDecodeShape{kWarpsPerSm >> i, 1 << j, rounds, segs * warps};
            }
        }
    }
    return out->warps ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_window_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const void* q,
                                 const int32_t* tables, const int32_t* seq_lens, void* out, int* err, int B,
                                 int Hq, int Hkv, int D, int block_size, int max_blocks, int num_blocks,
                                 int max_seq_len, float scale_log2, int window, int sinks, int out_bf16,
                                 int nslices, int GS, const WindowDecodeShape& shape, cudaStream_t stream) {
    WindowDecodeArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.tables = tables;
    a.seq_lens = seq_lens;
    a.out = out;
    a.err = err;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.nslices = nslices;
    a.GS = GS;
    a.U = Hkv * nslices;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.max_seq_len = max_seq_len;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = scale_log2;
    a.out_bf16 = out_bf16;
    a.probe_wait = wait_probe();
    a.cluster = shape.cluster;
    const int64_t blocks = static_cast<int64_t>(B) * a.U * shape.cluster;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto fn = select_window_decode(D, block_size, (GS + 7) / 8);
    const size_t smem = smem_bytes(shape.warps, GS, D);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cluster_launch(&cfg, attr, shape.cluster, 32 * shape.warps, smem);
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.stream = stream;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, a);
}

}  // namespace pa
