// Sliding-window attention with sinks for many queries (pa_prefill_window), on
// the tcgen05 tensor cores: a persistent kernel over a list of work items.
//
// The query at position p of a sequence attends to the tokens t <= p with
// p - t < W or t < S. A query tile holds 128 rows = (128 / g) queries x the g
// query heads of a kv head, and an item is two adjacent tiles of a sequence and
// kv head that share one K/V stream: the visible indices (WindowView) of their
// rows, in 128-token chunks through the block table. With a window an item is
// short whatever the prompt's length -- (W + S) / 128 chunks and one or two more
// -- so a block per item spends a good part of its time filling and draining
// its pipeline: 12 us of 39 at W = 2048 (two tiles of 17 chunks). Here one block
// per SM walks over its items and the pipeline runs on across them: the K and V
// copies are always a ring's depth ahead, the next item's queries are copied as
// soon as the last score product of the item has read its own, and its first
// score products are issued right behind the last value products. What is left
// between items is the read-out of O, one tile at a time, while the tensor core
// works on the other.
//
// Warps:
//   * 0-7 / 8-15 (softmax of tile 0 / 1): two threads a row, 64 of a chunk's
//     128 scores each, tensor memory read in the 16-lane shape so that both
//     sit in one warp. Scale to the log2 domain, mask by predicate (only the
//     chunks that an end of the window or the sinks' end cuts), row maximum,
//     P = 2^(s - m) as bf16 over the scores' first 64 columns. The running
//     maximum is raised only when a chunk exceeds it by more than 2^8 (any
//     reference gives the same quotient; this one bounds P by 256), and only
//     then is O rescaled. P is rounded to bf16 (8 bits) for the value product
//     while the row sum takes it unrounded, in 32 bits.
//   * 16, 18: tiled bulk tensor copies of K (with the query tiles) and V.
//   * 17: one thread issues, for every chunk and tile, O_t (+)= P_t V and then
//     S_t = Q_t K^T of the next chunk, or of the next item's first one. One
//     thread's products run in issue order, so a score product overwrites P_t
//     only after the value product has read it.
//   * 19: zeroes the value rows that no query of the item sees (between the
//     sinks and the first query's window, past the last query) in shared
//     memory, so that nothing hidden reaches a sum.
//
// The items come from window_items_kernel: sequences in order of length, their
// last tiles first, lengths and table entries validated once for all heads. Items
// go to blocks in turn. With few turns of long items, and at most half of the
// blocks at work in the last, a second build of the kernel (PARTS) cuts the last
// turn's items into parts by keys, one block a part: every warp leaves its 16
// rows' (m, l, O) of the part in memory and counts up, and the last to arrive
// merges them in the order of the parts, with m = max m_i, l = sum l_i 2^(m_i -
// m), o = sum O_i 2^(m_i - m) / l. No warp waits for another.
//
// What bounds it: the tensor cores are busy 68 % of the time. A tile's chain (its
// value products 512 cycles, its next score products 512, its softmax 1200, the
// hand-overs) is 2500 cycles a chunk against 2048 of products for both tiles, and
// an item's end costs 2500 to 5000 more: 16384 rows of W = 4096 612 us, 1593
// TFLOP/s (in passes apart; 655 to 662 us back to back at the power cap); 16 x 256
// rows of W = 2048 101.5 us, 1093 TFLOP/s (3.4 rounds of items in four). With two to
// six chunks an item its end is a third to a half of the time: 4 x 4096 rows of W =
// 128 89 us against 49 for the bytes, of 32 heads without groups, W = 512, 192
// against 79. So the code beside the softmax's loop counts: with its spills to
// local memory, which does not stay in what the rings leave of L1, and O stored
// by rows, the first took 691 us and the last 125.
//
// Every mbarrier wait is bounded. A role that gives up raises a shared abort
// flag (and PA_DEVERR_TIMEOUT); the others see it in their own waits. Before
// the block leaves, the copy warps wait (bounded) for their copies in flight,
// the MMA thread for its products, and the block frees its tensor memory.
#include <cuda_bf16.h>

#include <algorithm>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;      // M: query rows per tile
constexpr int kChunk = 128;     // tokens per K/V chunk
constexpr int kD = 128;         // head dimension
constexpr int kStagesK = 3;     // K ring depth
constexpr int kStagesV = 2;     // V ring depth
constexpr int kTileThreads = 2 * kRows;             // softmax threads of a tile: two per row
constexpr int kSoftmaxThreads = 2 * kTileThreads;
constexpr int kWarpLoad = kSoftmaxThreads / 32;     // warp 16: Q and K copies
constexpr int kWarpMma = kWarpLoad + 1;
constexpr int kWarpLoadV = kWarpMma + 1;
constexpr int kWarpZero = kWarpLoadV + 1;           // zeroes hidden value rows
constexpr int kThreads = kSoftmaxThreads + 128;
constexpr int kSortMax = 256;   // sequences ordered by length up to this batch size
constexpr uint32_t kTmemCols = 512;
// Tensor-memory columns: S of tile t (128; P_t over its first 64), then O of tile t (128).
__host__ __device__ constexpr uint32_t col_s(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * t; }
constexpr float kRescaleLog2 = 8.f;
constexpr int kMaxParts = 4;       // of an item of the last turn
constexpr int kMinPartChunks = 8;  // chunks a part
constexpr int kWarpsPerItem = kSoftmaxThreads / 32;
// A part's partial results: O [tile x 8 + warp][32 columns][register / 4][lane],
// as the warps read it for the output, then (m, l) of every row.
constexpr size_t kPartFloats = 2 * kRows * (kD + 2);

// Shared-memory layout (byte offsets from a 1024-aligned base).
constexpr uint32_t kTileQ = 32768;                    // 2 halves x 128 rows x 128 B
constexpr uint32_t kHalfKV = kChunk * 128;            // one 64-column half of a chunk
constexpr uint32_t kStageKV = 2 * kHalfKV;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kTileQ;
constexpr uint32_t kOffV = kOffK + kStagesK * kStageKV;
constexpr uint32_t kOffBar = kOffV + kStagesV * kStageKV;
// mbarriers (8 bytes each) and slots, at kOffBar + ...
constexpr uint32_t kBarKFull = 0;                          // [kStagesK]
constexpr uint32_t kBarKEmpty = kBarKFull + 8 * kStagesK;
constexpr uint32_t kBarVFull = kBarKEmpty + 8 * kStagesK;  // [kStagesV]
constexpr uint32_t kBarVEmpty = kBarVFull + 8 * kStagesV;
constexpr uint32_t kBarS = kBarVEmpty + 8 * kStagesV;      // [tile] scores ready
constexpr uint32_t kBarP = kBarS + 16;                     // [tile] P stored, kTileThreads arrivals
constexpr uint32_t kBarO = kBarP + 16;                     // [tile] an item's last value product done
constexpr uint32_t kBarQFull = kBarO + 16;                 // [tile] queries landed
constexpr uint32_t kBarQEmpty = kBarQFull + 16;            // [tile] an item's last score product done
constexpr uint32_t kBarDrain = kBarQEmpty + 16;
constexpr uint32_t kBarProbe = kBarDrain + 8;              // nothing completes it (wait-expiry probe)
constexpr uint32_t kSlotTmem = kBarProbe + 8;
constexpr uint32_t kSlotAbort = kSlotTmem + 4;
constexpr uint32_t kSlotItem = 256;                        // [softmax warp] 32 bytes: its item, while it goes over the chunks
constexpr uint32_t kSmemBytes = 1024 + kOffBar + kSlotItem + 32 * (kSoftmaxThreads / 32);
static_assert(kSlotAbort + 4 <= kSlotItem, "barrier area");
static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0, "swizzle atoms");
static_assert(kSmemBytes <= 227 * 1024 && 2 * kSmemBytes > 228 * 1024,
              "one block per SM: it holds all 512 tensor-memory columns");

constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kRows, kChunk, false, false);
constexpr uint32_t kIdescO = tc::idesc_bf16_f32(kRows, kD, false, true);  // B (V) MN-major

// Up to two query tiles of a sequence, for every kv head.
struct Item {
    int b;      // sequence
    int row;    // first query row (of q and out)
    int nq;     // queries (at most 2 x 128 / g); 0: nothing to do
    int pos;    // position of the first query
    int skip;   // pages left out between the sinks and the window
    int len;    // visible indices up to the last query
    int lo;     // first visible index within the first query's window
    int pad;
};

struct Args {
    const int32_t* q_start;
    const int32_t* tables;
    const int32_t* seq_lens;
    Item* items;
    int* num_items;
    int* arrived;             // [blocks][kWarpsPerItem] parts done, of the item whose first part is the block's
    float* parts;             // [blocks][kPartFloats]; null: no parts
    void* out;
    int* err;
    int B, Hq, Hkv, g, Qb;    // Qb = queries per tile = 128 / g
    int num_q, max_q, max_items;
    int max_blocks, num_blocks, max_seq_len;
    int window, sinks;
    float scale_log2;
    int out_bf16, probe_wait;
    int num_sms;
    int lg;                   // g = 2^lg (it divides 128)
};

// ------------------------------------------------------------------ items

constexpr int kItemThreads = 256;

// Zeroes output rows [r0, r1), all heads, the given threads in turn.
__device__ void zero_rows(const Args& a, int64_t r0, int64_t r1, int tid, int threads) {
    const int64_t per_row = static_cast<int64_t>(a.Hq) * kD;
    for (int64_t i = r0 * per_row + tid; i < r1 * per_row; i += threads) {
        if (a.out_bf16) static_cast<uint16_t*>(a.out)[i] = 0;
        else static_cast<float*>(a.out)[i] = 0.f;
    }
}

// The item list: every block orders the sequences and scans their item counts,
// its warps then fill items in turn (one item a warp: its table entries are
// checked by the lanes). Shared memory: pre[B + 1], then order[B].
template <int BS>
__global__ void __launch_bounds__(kItemThreads) window_items_kernel(const Args a) {
    extern __shared__ int sm[];
    __shared__ int warp_sums[kItemThreads / 32];
    int* pre = sm;
    int* order = sm + a.B + 1;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int limit = min(a.max_seq_len, a.max_blocks * BS);
    if (a.parts)
        for (int i = blockIdx.x * kItemThreads + tid; i < a.num_sms * kWarpsPerItem; i += gridDim.x * kItemThreads)
            a.arrived[i] = 0;
    // The items of sequence b: -1 if its lengths are wrong.
    auto count = [&](int b) {
        const int64_t qs = a.q_start[b], n = static_cast<int64_t>(a.q_start[b + 1]) - qs;
        const int L = a.seq_lens[b];
        if (n == 0) return 0;  // a request without queries in this step
        if (n < 1 || n > a.max_q || L < n || L > limit || qs < 0 || qs + n > a.num_q) return -1;
        return min(static_cast<int>((n + 2 * a.Qb - 1) / (2 * a.Qb)), a.max_items + 1);
    };
    // Longest sequence first (ties by index) when the batch is small enough.
    if (a.B <= kSortMax) {
        for (int i = tid; i < a.B; i += kItemThreads) pre[i] = a.seq_lens[i];
        __syncthreads();
        for (int i = tid; i < a.B; i += kItemThreads) {
            int r = 0;
            for (int j = 0; j < a.B; ++j) r += pre[j] > pre[i] || (pre[j] == pre[i] && j < i);
            order[r] = i;
        }
    } else {
        for (int i = tid; i < a.B; i += kItemThreads) order[i] = i;
    }
    __syncthreads();
    const int per = (a.B + kItemThreads - 1) / kItemThreads;
    const int lo = min(tid * per, a.B), hi = min(lo + per, a.B);
    int sum = 0;
    for (int r = lo; r < hi; ++r) {
        const int b = order[r], n = count(b);
        if (n < 0 && blockIdx.x == 0) atomicOr(a.err, kErrSeqLen);
        // The list holds the items of any nondecreasing q_start. The counts of
        // another are cut (here, so that they stay within 32 bits, and below),
        // and an item outside its sequence is dropped.
        sum = min(sum + max(n, 0), a.max_items + 1);
    }
    int x = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int run = x - sum;
    for (int w = 0; w < warp; ++w) run += warp_sums[w];
    for (int r = lo; r < hi; ++r) {
        pre[r] = run;
        run += max(count(order[r]), 0);
    }
    if (tid == kItemThreads - 1) pre[a.B] = run;
    __syncthreads();
    const int total = min(pre[a.B], a.max_items);
    if (blockIdx.x == 0 && tid == 0) {
        *a.num_items = total;
        if (pre[a.B] > a.max_items) atomicOr(a.err, kErrSeqLen);
    }
    // Rows of wrong sequences (those inside the arrays) become zeros.
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (count(b) >= 0) continue;
        const int64_t qs = a.q_start[b], qe = a.q_start[b + 1];
        zero_rows(a, max(qs, int64_t{0}), min(qe, static_cast<int64_t>(a.num_q)), tid, kItemThreads);
    }
    const int warps = gridDim.x * (kItemThreads / 32);
    for (int e = blockIdx.x * (kItemThreads / 32) + warp; e < total; e += warps) {
        int l = 0, h = a.B - 1;  // the last rank whose items start at or before e
        while (l < h) {
            const int mid = (l + h + 1) >> 1;
            if (pre[mid] <= e) l = mid; else h = mid - 1;
        }
        const int b = order[l];
        const int qs = a.q_start[b], n = a.q_start[b + 1] - qs, L = a.seq_lens[b];
        const int q0 = (pre[l + 1] - 1 - e) * 2 * a.Qb;  // the last tiles first: they see the most
        Item it;
        it.b = b;
        it.row = qs + q0;
        it.nq = q0 >= 0 ? max(0, min(2 * a.Qb, n - q0)) : 0;
        if (it.nq == 0) {
            if (lane == 0) {
                a.items[e] = Item{};
                atomicOr(a.err, kErrSeqLen);
            }
            continue;
        }
        it.pos = L - n + q0;
        const WindowView v = window_view(it.pos, it.pos + it.nq - 1, a.window, a.sinks, BS);
        it.skip = v.skip;
        it.len = v.len;
        it.lo = v.lo;
        it.pad = 0;
        const int32_t* table = a.tables + static_cast<size_t>(b) * a.max_blocks;
        const int sink_pages = (a.sinks + BS - 1) / BS;
        bool bad = false;
        for (int p = lane; p < (v.len + BS - 1) / BS; p += 32) {
            const int phys = table[p < sink_pages ? p : p + v.skip];
            bad |= phys < 0 || phys >= a.num_blocks;
        }
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) atomicOr(a.err, kErrTable);
            zero_rows(a, it.row, it.row + it.nq, lane, 32);
            it.nq = 0;
        }
        if (lane == 0) a.items[e] = it;
    }
}

// ------------------------------------------------------------------ attention

// Words j of threads 4 r .. 4 r + 3 become thread 4 r + j's: a 4 x 4 transpose.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4], int lane) {
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool odd = lane & bit;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = bit == 1 ? 2 * i : i;   // w[j] and w[j + bit]
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[j] : w[j + bit], bit);
            (odd ? w[j] : w[j + bit]) = got;
        }
    }
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Bounded wait that also gives up when another role raised the abort flag.
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, uint32_t abort_flag, int* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (ld_shared_u32(abort_flag)) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            st_shared_u32(abort_flag, 1);
            atomicOr(err, kErrTimeout);
            return false;
        }
    }
}

// The end of an item's part for the 16 rows of a warp: their (m, l, O) go to
// memory. True for the warp that is the last of the item's parts to do so: with
// the weights 2^(m_i - max m) of row lane & 15 in the parts, in their order, and
// the reciprocal of its sum. No warp waits for another.
__device__ __forceinline__ bool leave_part(const Args& a, uint32_t o_addr, float m, float lt, int part,
                                           float (&weight)[kMaxParts], float* inv) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* mine = a.parts + blockIdx.x * kPartFloats;
#pragma unroll
    for (int piece = 0; piece < 4; ++piece) {
        float o[16];
        tc::ld16x256_4(o_addr + 32 * piece, o);
        tc::wait_ld();
        float4* to = reinterpret_cast<float4*>(mine) + (warp * 4 + piece) * 128 + lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) __stcg(to + 32 * k, make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
    }
    tc::fence_before_sync();
    const size_t ml = 2 * kRows * kD + 2 * (warp * 16 + (lane & 15));
    if (lane < 16) __stcg(reinterpret_cast<float2*>(mine + ml), make_float2(m, lt));
    __threadfence();
    __syncwarp();
    const int parts = part & 7;
    int before = 0;
    if (lane == 0) before = atomicAdd(a.arrived + (part >> 3) * kWarpsPerItem + warp, 1);
    if (__shfl_sync(0xffffffffu, before, 0) != parts - 1) return false;
    __threadfence();
    const float* first = a.parts + (part >> 3) * kPartFloats + ml;
    float l[kMaxParts], mm = -INFINITY, lm = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
        const float2 v = i < parts ? __ldcg(reinterpret_cast<const float2*>(first + i * kPartFloats))
                                   : make_float2(-INFINITY, 0.f);
        weight[i] = v.x;
        l[i] = v.y;
    }
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) mm = fmaxf(mm, weight[i]);
    if (mm == -INFINITY) mm = 0.f;   // a row that sees nothing: its sums are 0
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
        weight[i] = fast_exp2(weight[i] - mm);
        lm += l[i] * weight[i];
    }
    *inv = lm > 0.f ? 1.f / lm : 0.f;
    return true;
}

// 32 columns of the merged O, as tc::ld16x256_4 gives them.
__device__ __forceinline__ void merge_parts(const Args& a, int part, int piece, const float (&weight)[kMaxParts],
                                            float (&o)[16]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float4* from = reinterpret_cast<const float4*>(a.parts + (part >> 3) * kPartFloats) + (warp * 4 + piece) * 128 + lane;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxParts; ++i) {
        if (i >= (part & 7)) break;
        const float w0 = __shfl_sync(0xffffffffu, weight[i], lane >> 2);
        const float w1 = __shfl_sync(0xffffffffu, weight[i], (lane >> 2) + 8);
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __ldcg(from + i * (kPartFloats / 4) + 32 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o[4 * k] += w0 * v[k].x;
            o[4 * k + 1] += w0 * v[k].y;
            o[4 * k + 2] += w1 * v[k].z;
            o[4 * k + 3] += w1 * v[k].w;
        }
    }
}

// This block's items in order: entry `turn * grid + block` of the list x kv heads
// (the heads of an item next to each other, so that running blocks share K/V
// pages in L2). PARTS: the items of a last, incomplete turn are cut into up to
// kMaxParts parts where the blocks suffice, block u * cut + i has part i of the
// turn's item u.
template <bool PARTS>
struct Walk {
    const Args& a;
    int total, turn;
    Item it;
    int h, c0, nc;  // kv head, first chunk, chunks
    int part;       // 0: the whole item; else its number of parts, and 8 x the block of the first
    __device__ __forceinline__ Walk(const Args& args)
        : a(args), total(*args.num_items * args.Hkv), turn(-1), c0(0), part(0) {}
    __device__ __forceinline__ bool next() {
        const int grid = gridDim.x;
        while (true) {
            ++turn;
            const int left = total - turn * grid;   // from this turn on
            const int cut = PARTS && left > 0 && left < grid ? min(kMaxParts, grid / left) : 1;
            const int u = PARTS ? static_cast<int>(blockIdx.x) / cut : static_cast<int>(blockIdx.x);
            if (u >= left) return false;
            const int id = turn * grid + u;
            const int e = id / a.Hkv;
            const int4* p = reinterpret_cast<const int4*>(a.items + e);
            const int4 x = p[0], w = p[1];
            if (x.z == 0) continue;
            it = Item{x.x, x.y, x.z, x.w, w.x, w.y, w.z, 0};
            h = id - e * a.Hkv;
            nc = (it.len + kChunk - 1) / kChunk;
            if (PARTS) c0 = 0, part = 0;
            if (PARTS && cut > 1) {
                const int per = max(kMinPartChunks, (nc + cut - 1) / cut), parts = (nc + per - 1) / per;
                c0 = (blockIdx.x - u * cut) * per;
                if (parts > 1) part = parts + 8 * u * cut;
                nc = min(per, nc - c0);
                if (nc <= 0) continue;
            }
            return true;
        }
    }
};

template <int BS, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bars = base + kOffBar;
    const uint32_t abort_flag = bars + kSlotAbort;  // a shared-memory address: one register

    if (tid == 0) {
        for (int s = 0; s < kStagesK; ++s) {
            mbar_init(bars + kBarKFull + 8 * s, 1);
            mbar_init(bars + kBarKEmpty + 8 * s, 1);
        }
        for (int s = 0; s < kStagesV; ++s) {
            mbar_init(bars + kBarVFull + 8 * s, 1);
            mbar_init(bars + kBarVEmpty + 8 * s, 1);
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(bars + kBarS + 8 * u, 1);
            // Tile 0's also waits for the warp that zeroes value rows.
            mbar_init(bars + kBarP + 8 * u, kTileThreads + (u == 0 ? 1 : 0));
            mbar_init(bars + kBarO + 8 * u, 1);
            mbar_init(bars + kBarQFull + 8 * u, 1);
            mbar_init(bars + kBarQEmpty + 8 * u, 1);
        }
        mbar_init(bars + kBarDrain, 1);
        mbar_init(bars + kBarProbe, 1);
        st_shared_u32(abort_flag, 0);
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        prefetch_tensormap(&qmap);
    }
    if (warp == kWarpMma) {
        tc::alloc(bars + kSlotTmem, kTmemCols);
        tc::relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + kOffBar + kSlotTmem);
    griddep_wait();  // the item list, and whatever came before it
    griddep_launch_dependents();

    if (warp >= kWarpLoad) {

        if (warp == kWarpLoad || warp == kWarpLoadV) {
            // ------------------------------------------------------------ copies (Q and K, V)
            // The whole warp runs this loop and one thread issues, as below: from
            // one thread the 16 boxes of a chunk took 1,900 cycles.
            const uint32_t one = elect_one();
            const bool is_k = warp == kWarpLoad;
            const int nst = is_k ? kStagesK : kStagesV;
            const uint32_t full = bars + (is_k ? kBarKFull : kBarVFull);
            const uint32_t empty = bars + (is_k ? kBarKEmpty : kBarVEmpty);
            const uint32_t ring = base + (is_k ? kOffK : kOffV);
            const CUtensorMap* map = is_k ? &kmap : &vmap;
            const int sink_pages = (a.sinks + BS - 1) / BS;
            constexpr int kPages = kChunk / BS;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait_role(bar, parity, abort_flag, a.err)) != 0;
            };
            // K/V pages of an item are read again for the item's neighbours:
            // no eviction hint, unlike the kernels that read a page once.
            Walk<PARTS> w(a);
            int s = 0;                 // ring stage
            uint32_t parity = 1;       // of its last release: a fresh stage counts as released
            int issued = 0;            // chunks in the ring, at most nst
            uint32_t qp[2] = {1, 1};   // the query buffers, likewise
            int q_used = 0;            // bit u: buffer u holds or awaits a tile
            bool ok = true;
            while (ok && w.next()) {
                const int32_t* table = a.tables + static_cast<size_t>(w.it.b) * a.max_blocks;
                const int nb = __shfl_sync(0xffffffffu, (w.it.len + BS - 1) / BS, 0);
                const int nc = __shfl_sync(0xffffffffu, w.nc, 0), h = __shfl_sync(0xffffffffu, w.h, 0);
                const int c0 = PARTS ? __shfl_sync(0xffffffffu, w.c0, 0) : 0;
                // Lane j: the block of page j of chunk c, one chunk ahead.
                auto entries = [&](int c) {
                    const int p = (c0 + c) * kPages + lane;
                    return lane < kPages && p < nb ? table[p < sink_pages ? p : p + w.it.skip] : 0;
                };
                int pg = entries(0);
                for (int c = 0; c < nc; ++c) {
                    const int pg_next = c + 1 < nc ? entries(c + 1) : 0;
                    ok = wait(empty + 8 * s, parity);
                    if (!ok) break;
                    const int np = min(kPages, nb - (c0 + c) * kPages);
                    const uint32_t bar = full + 8 * s, stage = ring + s * kStageKV;
                    if (one) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np) * BS * kD * 2);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < kPages; ++j) {
                        const int r = __shfl_sync(0xffffffffu, pg, j) * a.Hkv + h;
                        const uint32_t on = j < np ? one : 0u;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_3d_if(on, stage + hf * kHalfKV + j * BS * 128, map, hf * 64, 0, r, bar);
                    }
                    pg = pg_next;
                    issued = min(issued + 1, nst);
                    if (++s == nst) s = 0, parity ^= 1u;
                    if (is_k && c == 0) {
                        // The item's queries behind its first keys (whose stage
                        // is free before the queries' buffer is): one box per
                        // 64-column half, rows in (query, head) order. Rows past
                        // the item's queries hold other rows of q or zeros; they
                        // are never stored.
                        const int row = __shfl_sync(0xffffffffu, w.it.row, 0);
                        const int tiles = __shfl_sync(0xffffffffu, w.it.nq > a.Qb ? 2 : 1, 0);
                        for (int u = 0; u < tiles && ok; ++u) {
                            ok = wait(bars + kBarQEmpty + 8 * u, qp[u]);
                            if (!ok) break;
                            qp[u] ^= 1u;
                            q_used |= 1 << u;
                            const uint32_t qbar = bars + kBarQFull + 8 * u;
                            if (one) mbar_arrive_expect_tx(qbar, kTileQ);
                            __syncwarp();
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
                                tma_load_3d_if(one, base + kOffQ + u * kTileQ + hf * 16384, &qmap, hf * 64, h * a.g,
                                               row + u * a.Qb, qbar);
                        }
                        if (!ok) break;
                    }
                }
            }
            // Copies still in flight land before the block leaves: the last
            // chunk issued on each stage and the last tile of each query
            // buffer. Without an abort their consumers have waited for them.
            for (int i = 0; i < issued; ++i) {
                if (--s < 0) s = nst - 1, parity ^= 1u;
                mbar_wait_bounded(full + 8 * s, parity ^ 1u, kWaitLimitNs);
            }
            if (is_k)
                for (int u = 0; u < 2; ++u)
                    if (q_used >> u & 1) mbar_wait_bounded(bars + kBarQFull + 8 * u, qp[u], kWaitLimitNs);
        } else if (warp == kWarpMma) {
            // ------------------------------------------------------------ products
            // The whole warp runs this loop and one thread issues: with the loop
            // in one thread every product took 87 cycles to issue, its operands
            // moved to uniform registers each time.
            const uint32_t one = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t hi = static_cast<uint32_t>(tc::smem_desc(base, 16, 1024) >> 32);
            const uint32_t lo_q = tc::desc_lo(base + kOffQ, 16);
            const uint32_t lo_k = tc::desc_lo(base + kOffK, 16);
            const uint32_t lo_v = tc::desc_lo(base + kOffV, kHalfKV);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                const bool ok = __all_sync(0xffffffffu, wait_role(bars + bar, parity, abort_flag, a.err));
                tc::fence_after_sync();
                return ok;
            };
            // S_u of the chunk in K stage s.
            auto issue_s = [&](int u, int s) {
                const uint32_t a0 = lo_q + u * (kTileQ >> 4), b0 = lo_k + s * (kStageKV >> 4);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t da = (kk >> 2) * (16384 >> 4) + (kk & 3) * 2;
                    const uint32_t db = (kk >> 2) * (kHalfKV >> 4) + (kk & 3) * 2;
                    tc::mma_bf16_lo_if(one, tm + col_s(u), a0 + da, b0 + db, hi, kIdescS, kk > 0);
                }
                tc::commit_if(one, bars + kBarS + 8 * u);
            };
            // O_u (+)= P_u V of the chunk in V stage s.
            auto issue_pv = [&](int u, int s, uint32_t add) {
                const uint32_t b0 = lo_v + s * (kStageKV >> 4);
#pragma unroll
                for (int kk = 0; kk < kChunk / 16; ++kk)   // 16 tokens = 8 columns of P
                    tc::mma_bf16_ts_if(one, tm + col_o(u), tm + col_s(u) + kk * 8, b0 + kk * (2048 >> 4), hi,
                                       kIdescO, kk > 0 ? 1u : add);
            };
            bool ok = true;
            if (a.probe_wait) {
                // The wait-expiry probe: a bounded wait on a barrier nothing
                // completes, then the abort every other role follows.
                mbar_wait_bounded(bars + kBarProbe, 0, kProbeLimitNs);
                st_shared_u32(abort_flag, 1);
                if (lane == 0) atomicOr(a.err, kErrTimeout);
                ok = false;
            }
            Walk<PARTS> w(a);
            // Ring stages and parities of the chunk whose value products come
            // next, and of the chunk whose score products do; parities of P and
            // of the query tiles.
            int vs = 0, ks = 0;
            uint32_t vp = 0, kp = 0, pp[2] = {0, 0}, qp[2] = {0, 0};
            int nc = 0, two = 0;                 // the item whose scores come next
            auto next_item = [&] {
                const bool more = w.next();
                nc = __shfl_sync(0xffffffffu, more ? w.nc : 0, 0);
                two = __shfl_sync(0xffffffffu, more && w.it.nq > a.Qb ? 1 : 0, 0);
            };
            auto value_products = [&](int u, uint32_t add) {
                if (!wait(kBarP + 8 * u, pp[u])) return false;
                pp[u] ^= 1u;
                issue_pv(u, vs, add);
                return true;
            };
            auto query_tile = [&](int u) {       // an item's first score product of tile u
                const bool ok = wait(kBarQFull + 8 * u, qp[u]);
                qp[u] ^= 1u;
                return ok;
            };
            if (ok) next_item();
            if (ok && nc > 0) {
                ok = query_tile(0) && wait(kBarKFull, 0);
                if (ok) {
                    issue_s(0, 0);
                    if (nc == 1) tc::commit_if(one, bars + kBarQEmpty);
                    if (two && (ok = query_tile(1))) {
                        issue_s(1, 0);
                        if (nc == 1) tc::commit_if(one, bars + kBarQEmpty + 8);
                    }
                    tc::commit_if(one, bars + kBarKEmpty);
                    ks = 1;
                }
            }
            while (ok && nc > 0) {
                const int n = nc, pair = two;    // the item whose value products come next
                for (int c = 0; c < n; ++c) {
                    const bool end = c + 1 == n;
                    if (end) next_item();
                    const bool more = nc > 0;
                    // The last score products of their item free its queries.
                    const bool last = end ? nc == 1 : c + 2 == n;
                    // What the products need besides P is there by now; P comes
                    // last, so that nothing is waited for between them.
                    ok = wait(kBarVFull + 8 * vs, vp) && (!more || wait(kBarKFull + 8 * ks, kp)) &&
                         value_products(0, c > 0);
                    if (!ok) break;
                    if (end) tc::commit_if(one, bars + kBarO);
                    if (more) {
                        ok = !end || query_tile(0);
                        if (!ok) break;
                        issue_s(0, ks);
                        if (last) tc::commit_if(one, bars + kBarQEmpty);
                    }
                    if (pair) {
                        ok = value_products(1, c > 0);
                        if (!ok) break;
                        if (end) tc::commit_if(one, bars + kBarO + 8);
                    }
                    tc::commit_if(one, bars + kBarVEmpty + 8 * vs);
                    if (more) {
                        if (two) {
                            ok = !end || query_tile(1);
                            if (!ok) break;
                            issue_s(1, ks);
                            if (last) tc::commit_if(one, bars + kBarQEmpty + 8);
                        }
                        tc::commit_if(one, bars + kBarKEmpty + 8 * ks);
                        if (++ks == kStagesK) ks = 0, kp ^= 1u;
                    }
                    if (++vs == kStagesV) vs = 0, vp ^= 1u;
                }
            }
            // Every product is done before the block leaves.
            tc::commit_if(one, bars + kBarDrain);
            mbar_wait_bounded(bars + kBarDrain, 0, kWaitLimitNs);
        } else if (warp == kWarpZero) {
            // ------------------------------------------------------------ hidden value rows
            // Rows of V that no query of the item sees (between the sinks and
            // the first query's window, and past the last query) become zeros
            // before the chunk's value products: this warp's arrival is one of
            // those that tile 0's P waits for. It arrives once a chunk, after
            // S_0 of the chunk, so never for a later one. The wait for V is
            // unambiguous: S_0 of this step was issued after the value product
            // of the step before, which waited for that step's V.
            Walk<PARTS> w(a);
            int step = 0;
            bool ok = true;
            while (ok && w.next()) {
                for (int c = 0; c < w.nc; ++c, ++step) {
                    ok = __all_sync(0xffffffffu, wait_role(bars + kBarS, step & 1, abort_flag, a.err));
                    if (!ok) break;
                    const int v0 = (w.c0 + c) * kChunk;
                    const int h0 = max(0, a.sinks - v0), h1 = min(kChunk, w.it.lo - v0);
                    const int valid = min(kChunk, w.it.len - v0);
                    if (valid < kChunk || h0 < h1) {
                        ok = __all_sync(0xffffffffu, wait_role(bars + kBarVFull + 8 * (step % kStagesV),
                                                               (step / kStagesV) & 1, abort_flag, a.err));
                        if (!ok) break;
                        const uint32_t vst = base + kOffV + (step % kStagesV) * kStageKV + (lane >> 3 & 1) * kHalfKV +
                                             (lane & 7) * 16;
                        for (int r = h0 + (lane >> 4); r < h1; r += 2)
                            st_shared_v4(vst + r * 128, make_uint4(0, 0, 0, 0));
                        for (int r = valid + (lane >> 4); r < kChunk; r += 2)
                            st_shared_v4(vst + r * 128, make_uint4(0, 0, 0, 0));
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(bars + kBarP);
                }
            }
        }
        __syncwarp();
    } else {

        // ------------------------------------------------------------ softmax (tile t)
        // The 8 warps of a tile cover its 128 tensor-memory lanes in 16-lane
        // groups, each within its lane quarter; threads i and i + 16 of a warp
        // share a row, each on 64 of its scores (half).
        const int t = tid / kTileThreads;
        const int half = lane >> 4;
        const int row = 32 * (warp & 3) + 16 * ((warp >> 2) & 1) + (lane & 15);
        const uint32_t lane_base = static_cast<uint32_t>(row & ~15) << 16;
        const uint32_t s_addr = tmem + lane_base + col_s(t);
        const uint32_t o_addr = s_addr + (col_o(0) - col_s(0));
        static_assert(col_o(1) - col_s(1) == col_o(0) - col_s(0), "columns");
        const int qi = row >> a.lg;
        Walk<PARTS> w(a);
        bool ok = true;
        uint32_t phase = 0;   // parities: bit 0 of the scores' barrier, bit 1 of the output's
        while (ok && w.next()) {
            const int nq_t = w.it.nq - t * a.Qb;  // queries of this tile
            if (nq_t <= 0) continue;
            const int nc = w.nc;
            // Indices count from the part's first chunk on. The last that the
            // tile's first query sees:
            const int pos_t = w.it.pos + t * a.Qb - w.it.skip * BS - w.c0 * kChunk;
            const int pos_r = pos_t + qi;                            // ... and this row's
            // The chunks that need a mask for some query of this warp (rows past
            // the tile's queries are never stored and need none): from c_hi on
            // those that its first query's position cuts, and c_lo0 .. c_lo1
            // those between the sinks and its last query's window.
            const int qa = ((row & ~15) >> a.lg), qb = min((row | 15) >> a.lg, nq_t - 1);
            const int c_hi = qa < nq_t ? (pos_t + qa + 1) / kChunk : nc;
            const int sinks = a.sinks - w.c0 * kChunk;
            const int c_lo0 = sinks / kChunk;
            const int c_lo1 = qa < nq_t && pos_t + qb >= a.window ? (pos_t + qb - a.window) / kChunk : -1;
            // What only the end of the item needs waits in shared memory: with
            // it in registers the compiler spilled, to local memory that does
            // not stay in the 28 KB of L1 left beside the rings.
            const uint32_t slot = bars + kSlotItem + 32 * warp;
            if (lane == 0) {
                st_shared_v4(slot, make_uint4(w.turn, w.total, w.it.row, nq_t | w.h << 16));
                if (PARTS) st_shared_u32(slot + 16, w.part);
            }
            __syncwarp();
            float m = -INFINITY, l = 0.f;
            for (int c = 0; c < nc; ++c) {
                // S_t(c) done; its commit also covers the value product before it.
                ok = __all_sync(0xffffffffu, wait_role(bars + kBarS + 8 * t, phase & 1u, abort_flag, a.err));
                if (!ok) break;
                phase ^= 1u;
                tc::fence_after_sync();
                float sv[kChunk / 2];
                tc::ld16x2_32<64>(s_addr, *reinterpret_cast<float(*)[32]>(sv));
                tc::ld16x2_32<64>(s_addr + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
                tc::wait_ld();
                if (c >= c_hi) {
                    const int last = pos_r - c * kChunk - 64 * half;
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i) sv[i] = i <= last ? sv[i] : -INFINITY;
                }
                if (c >= c_lo0 && c <= c_lo1) {
                    const int h0 = sinks - c * kChunk - 64 * half, h1 = pos_r - a.window - c * kChunk - 64 * half;
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i) sv[i] = (i < h0 || i > h1) ? sv[i] : -INFINITY;
                }
                // Row max: three-input max over pairs, four short chains, then the
                // partner's half.
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kChunk / 4; ++i) mq[i & 3] = max3(mq[i & 3], sv[2 * i], sv[2 * i + 1]);
                float mx = max3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                mx *= a.scale_log2;  // scale > 0: the max of the scaled scores
                float alpha = 1.f;
                if (mx > m + kRescaleLog2) {
                    alpha = fast_exp2(m - mx);  // 0 while m is still -inf
                    m = mx;
                    l *= alpha;
                }
                // Rescale this row's half of O_t if its reference max moved.
                if (c > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1  // rare, and short code keeps the rest in the instruction cache
                    for (int piece = 0; piece < 8; ++piece) {
                        float o[8];
                        tc::ld16x2_8<64>(o_addr + 8 * piece, o);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] *= alpha;
                        tc::st16x2_8<64>(o_addr + 8 * piece, o);
                    }
                }
                const float m_use = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = f32x2(a.scale_log2, a.scale_log2), nm2 = f32x2(-m_use, -m_use);
                uint64_t ps2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t pw[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = f32x2_split(
                            fma_f32x2(f32x2(sv[32 * h2 + 2 * i], sv[32 * h2 + 2 * i + 1]), sc2, nm2));
                        const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                        ps2[i & 1] = add_f32x2(ps2[i & 1], f32x2(p0, p1));
                        pw[i] = pack_bf16x2(p0, p1);
                    }
                    tc::st16x2_16u<32>(s_addr + 16 * h2, pw);
                }
                tc::wait_st();
                tc::fence_before_sync();
                mbar_arrive(bars + kBarP + 8 * t);
                const float2 s0 = f32x2_split(ps2[0]), s1 = f32x2_split(ps2[1]);
                l += (s0.x + s0.y) + (s1.x + s1.y);
            }
            if (!ok) break;
            // The item's rows: O_t normalised, stored by the threads (the query
            // buffer already takes the next item's queries).
            ok = __all_sync(0xffffffffu, wait_role(bars + kBarO + 8 * t, phase >> 1, abort_flag, a.err));
            if (!ok) break;
            phase ^= 2u;
            tc::fence_after_sync();
            const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);
            float inv = lt > 0.f ? 1.f / lt : 0.f;
            const uint4 kept = ld_shared_v4(slot);
            w.turn = kept.x;
            w.total = kept.y;
            int part = 0;
            float weight[kMaxParts];  // of row lane & 15 in the parts
            if constexpr (PARTS) {
                part = ld_shared_u32(slot + 16);
                if (part && !leave_part(a, o_addr, m, lt, part, weight, &inv)) continue;
            }
            // Four threads a row, 32 columns of two rows at a time, so that a
            // store of the warp covers 8 rows by 64 bytes. (Rows as the softmax
            // holds them, 16 bytes of 32 places a store, kept the stores' path
            // busy for 4000 cycles an item and all loads behind them waiting.)
            const int nq_end = kept.w & 0xffff;
            const int ra = (row & ~15) + (lane >> 2), qa0 = ra >> a.lg, qa1 = (ra + 8) >> a.lg;
            const float inv0 = __shfl_sync(0xffffffffu, inv, lane >> 2);
            const float inv1 = __shfl_sync(0xffffffffu, inv, (lane >> 2) + 8);
            const size_t first = (static_cast<size_t>(kept.z) + t * a.Qb) * a.Hq + (kept.w >> 16) * a.g;
            const size_t at0 = (first + static_cast<size_t>(qa0) * a.Hq + (ra & (a.g - 1))) * kD;
            const size_t at1 = (first + static_cast<size_t>(qa1) * a.Hq + ((ra + 8) & (a.g - 1))) * kD;
#pragma unroll
            for (int piece = 0; piece < 4; ++piece) {
                float o[16];
                if (PARTS && part) {
                    merge_parts(a, part, piece, weight, o);
                } else {
                    tc::ld16x256_4(o_addr + 32 * piece, o);
                    tc::wait_ld();
                }
                if (a.out_bf16) {
                    uint32_t w0[4], w1[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w0[j] = pack_bf16x2(o[4 * j] * inv0, o[4 * j + 1] * inv0);
                        w1[j] = pack_bf16x2(o[4 * j + 2] * inv1, o[4 * j + 3] * inv1);
                    }
                    transpose4(w0, lane);
                    transpose4(w1, lane);
                    uint16_t* out = static_cast<uint16_t*>(a.out) + 32 * piece + 8 * (lane & 3);
                    if (qa0 < nq_end) *reinterpret_cast<uint4*>(out + at0) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
                    if (qa1 < nq_end) *reinterpret_cast<uint4*>(out + at1) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
                } else {
                    float* out = static_cast<float*>(a.out) + 32 * piece + 2 * (lane & 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (qa0 < nq_end)
                            *reinterpret_cast<float2*>(out + at0 + 8 * j) = make_float2(o[4 * j] * inv0, o[4 * j + 1] * inv0);
                        if (qa1 < nq_end)
                            *reinterpret_cast<float2*>(out + at1 + 8 * j) = make_float2(o[4 * j + 2] * inv1, o[4 * j + 3] * inv1);
                    }
                }
            }
            tc::fence_before_sync();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        tc::fence_after_sync();
        tc::dealloc(tmem, kTmemCols);
    }
}

int64_t items_bound(int B, int Hq, int Hkv, int64_t num_q) {
    const int64_t rows = 2 * (kRows / (Hq / Hkv));
    return (num_q + rows - 1) / rows + B;
}

}  // namespace

namespace {

// Whether a call runs the kernel that cuts its last turn's items (PARTS): few
// turns of long items, the last one filling at most half of the blocks (the
// number of items is a guess where the sequences' query counts differ; any other
// number is only slower). Leaving and merging the parts costs about 5 us, and the
// code beside the softmax 1 to 4 % of all turns. Measured, us, uncut and cut: 160
// items, W = 3300 94 and 77, W = 8192 202 and 146; 320 items 138 and 122; 624
// items 224 and 212; 768 items, five turns and 8, 266 and 269; W = 2048: 160
// items 64 and 62, 512 items 111 and 119. A last turn of more than half of the
// blocks is not cut: 448 items, W = 8192, 313 and 325.
bool cut_items(int Hq, int Hkv, int num_q, int vis_len, int num_sms) {
    const int rows = 2 * (kRows / (Hq / Hkv));
    const int64_t items = (static_cast<int64_t>(num_q) + rows - 1) / rows * Hkv;
    const int64_t left = items % num_sms;
    return vis_len >= 24 * kChunk && items < 5 * static_cast<int64_t>(num_sms) && left > 0 && 2 * left <= num_sms;
}

// The workspace: the item count (256 bytes), the items, and where items are cut
// the arrival counts and the partial results.
size_t item_bytes(int B, int Hq, int Hkv, int num_q) {
    return 256 + (static_cast<size_t>(items_bound(B, Hq, Hkv, num_q)) * sizeof(Item) + 255) / 256 * 256;
}

size_t arrived_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * kWarpsPerItem * 4 + 255) / 256 * 256; }

}  // namespace

size_t prefill_window_bytes(int B, int Hq, int Hkv, int num_q, int vis_len, int num_sms) {
    const size_t n = item_bytes(B, Hq, Hkv, num_q);
    if (!cut_items(Hq, Hkv, num_q, vis_len, num_sms)) return n;
    return n + arrived_bytes(num_sms) + num_sms * kPartFloats * 4;
}

cudaError_t launch_prefill_window(const CUtensorMap& kmap, const CUtensorMap& vmap, const void* q,
                                  int num_q, const int32_t* q_start, const int32_t* tables,
                                  const int32_t* seq_lens, void* out, int* err, int B, int Hq, int Hkv,
                                  int max_blocks, int num_blocks, int max_seq_len, int max_q,
                                  float scale_log2, int window, int sinks, int out_bf16, int block_size,
                                  int vis_len, int num_sms, void* ws, cudaStream_t stream) {
    Args a{};
    a.q_start = q_start;
    a.tables = tables;
    a.seq_lens = seq_lens;
    a.num_items = static_cast<int*>(ws);
    a.items = reinterpret_cast<Item*>(static_cast<char*>(ws) + 256);
    const bool cut = cut_items(Hq, Hkv, num_q, vis_len, num_sms);
    if (cut) {
        char* at = static_cast<char*>(ws) + item_bytes(B, Hq, Hkv, num_q);
        a.arrived = reinterpret_cast<int*>(at);
        a.parts = reinterpret_cast<float*>(at + arrived_bytes(num_sms));
    }
    a.num_sms = num_sms;
    a.out = out;
    a.err = err;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.Qb = kRows / a.g;
    a.lg = 0;
    while (1 << a.lg < a.g) ++a.lg;
    a.num_q = num_q;
    a.max_q = max_q;
    a.max_items = static_cast<int>(std::min<int64_t>(items_bound(B, Hq, Hkv, num_q), INT32_MAX / Hkv - num_sms));
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.max_seq_len = max_seq_len;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = scale_log2;
    a.out_bf16 = out_bf16;
    a.probe_wait = wait_probe();
    CUtensorMap qmap;
    if (!encode_query_map(&qmap, q, num_q, Hq, a.g, a.Qb)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(num_sms, (a.max_items + 7) / 8)));
    cfg.blockDim = dim3(kItemThreads);
    cfg.dynamicSmemBytes = (2 * static_cast<size_t>(B) + 1) * sizeof(int);
    auto items = block_size == 16 ? window_items_kernel<16> : window_items_kernel<32>;
    // The limit belongs to the function, which other threads launch with other
    // batches: that of the largest.
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(items),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>((2 * kMaxBatch + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, items, a);
    if (e != cudaSuccess) return e;
    auto kern = cut ? (block_size == 16 ? window_kernel<16, true> : window_kernel<32, true>)
                    : (block_size == 16 ? window_kernel<16, false> : window_kernel<32, false>);
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(
        cut ? num_sms : std::min<int64_t>(num_sms, static_cast<int64_t>(a.max_items) * Hkv)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, qmap, a);
}

}  // namespace pa
