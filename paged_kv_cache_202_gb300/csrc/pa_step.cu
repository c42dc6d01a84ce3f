// Step maps: block tables, lengths, query offsets and slots of a serving step,
// from the requests' cached lengths and new token counts.
//
// A request's tokens fill whole blocks in order, so a step that adds n tokens
// to c cached ones needs ceil((c + n) / bs) - ceil(c / bs) fresh blocks ("any
// free block fits any request", "PagedAttention: The Cache Was Storing
// Nothing" §2.2). With the exclusive prefix sums of n (the rows of a packed
// batch, q_start) and of the fresh blocks (places in the free list), every
// row's position, block and slot follow on their own: row t of request b sits
// at position p = c_b + t - q_start[b], in the table's block p / bs if that
// was there before, else in the fresh block number p / bs - ceil(c_b / bs) of
// the request. A row at the start of a block writes the table entry.
//
// One launch without any exchange between blocks: every block scans all
// requests in shared memory (two scans, B <= 8192 values each) and then takes
// its rows, so there is no second kernel to wait for. Entries read from the
// table (blocks the request had) and entries written (fresh ones) are
// different ones. The work is a few bytes a row; what bounds it is the launch
// and the latency of the dependent steps (lengths, scans, search, table
// entry): 64 decoding requests 3.1 us, of which about 2 are a launch; 1024
// requests with 261,000 rows 6.7 us, 8.1 with maps that are not in L2, 0.4 TB/s.
#include <algorithm>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kStepThreads = 512;

struct StepArgs {
    const int32_t* cache_lens;
    const int32_t* new_lens;
    const int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* tables;
    int32_t* seq_lens;
    int32_t* q_start;
    int32_t* positions;
    int64_t* slots;
    int32_t* free_left;
    int* err;
    int B, max_blocks, num_free, shift, num_blocks, limit, T;
};

// Exclusive scan of one 64-bit value per thread over the block; *total
// receives the sum. Every thread calls it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) {
        const int64_t s = warp_sums[w];
        before += w < warp ? s : 0;
        all += s;
    }
    __syncthreads();  // warp_sums may be written again
    *total = all;
    return before + x - v;
}

__global__ void __launch_bounds__(kStepThreads) step_maps_kernel(const StepArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int64_t warp_sums[kStepThreads / 32];
    int32_t* start = sm;                // [B + 1] rows before request b, at most T
    int32_t* fresh = sm + a.B + 1;      // [B] fresh blocks before request b, -1: no slots
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int bs = 1 << a.shift;
    const bool first = blockIdx.x == 0;
    const int per = (a.B + kStepThreads - 1) / kStepThreads;
    const int lo = min(tid * per, a.B), hi = min(lo + per, a.B);
    int count = *a.free_count;
    bool bad = false;
    const bool bad_count = count < 0 || count > a.num_free;
    if (bad_count) count = 0;

    // Rows before each request. A negative count of new tokens is no row.
    int64_t sum = 0, total;
    for (int b = lo; b < hi; ++b) sum += max(a.new_lens[b], 0);
    int64_t run = block_scan(sum, warp_sums, &total);
    // Fresh blocks of the valid requests: lengths within the table and the
    // limit, rows within T.
    int64_t need_sum = 0;
    for (int b = lo; b < hi; ++b) {
        const int n = a.new_lens[b], c = a.cache_lens[b];
        start[b] = static_cast<int32_t>(min(run, static_cast<int64_t>(a.T)));
        run += max(n, 0);
        const bool ok = n >= 0 && c >= 0 && static_cast<int64_t>(c) + n <= a.limit && run <= a.T;
        bad |= !ok;
        const int need = ok ? ((c + n + bs - 1) >> a.shift) - ((c + bs - 1) >> a.shift) : 0;
        fresh[b] = ok ? need : -1;
        need_sum += need;
    }
    if (tid == kStepThreads - 1) start[a.B] = static_cast<int32_t>(min(total, static_cast<int64_t>(a.T)));
    int64_t need_total;
    int64_t taken = block_scan(need_sum, warp_sums, &need_total);
    // All or nothing: with too few free blocks none is taken, and the requests
    // that needed one get no slots.
    const bool short_of = need_total > count;
    for (int b = lo; b < hi; ++b) {
        const int need = fresh[b];
        const bool ok = need == 0 || (need > 0 && !short_of);
        fresh[b] = ok ? static_cast<int32_t>(short_of ? 0 : taken) : -1;
        taken += max(need, 0);
        if (first) {
            a.seq_lens[b] = ok ? a.cache_lens[b] + a.new_lens[b] : 0;
            a.q_start[b] = start[b];
        }
    }
    __syncthreads();
    int flags = (bad ? kErrSeqLen : 0) | (bad_count ? kErrTable : 0);
    if (first && tid == 0) {
        a.q_start[a.B] = start[a.B];
        *a.free_left = count - (short_of ? 0 : static_cast<int32_t>(need_total));
        if (short_of) flags |= kErrNoBlocks;
    }
    if (!first) flags = 0;

    const int rows = start[a.B];
    for (int64_t t64 = static_cast<int64_t>(blockIdx.x) * kStepThreads + tid; t64 < a.T;
         t64 += static_cast<int64_t>(gridDim.x) * kStepThreads) {
        const int t = static_cast<int>(t64);
        int pos = 0;
        int64_t slot = -1;
        if (t < rows) {
            int l = 0, h = a.B - 1;  // the last request that starts at or before t
            while (l < h) {
                const int mid = (l + h + 1) >> 1;
                if (start[mid] <= t) l = mid; else h = mid - 1;
            }
            const int f = fresh[l];
            const int c = a.cache_lens[l];
            if (f >= 0) {
                pos = c + (t - start[l]);
                const int page = pos >> a.shift, had = (c + bs - 1) >> a.shift;
                int32_t* entry = a.tables + static_cast<size_t>(l) * a.max_blocks + page;
                int32_t phys;
                if (page < had) {
                    phys = *entry;
                } else {
                    phys = a.free_blocks[count - 1 - (f + page - had)];
                    if ((pos & (bs - 1)) == 0) *entry = phys;
                }
                if (phys >= 0 && phys < a.num_blocks)
                    slot = (static_cast<int64_t>(phys) << a.shift) + (pos & (bs - 1));
                else
                    flags |= kErrTable;
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    if (flags) atomicOr(a.err, flags);
}

}  // namespace
}  // namespace pa

namespace {

// Whether the n and m bytes at a and b share any.
bool overlap(const void* a, size_t n, const void* b, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
}

}  // namespace

extern "C" pa_status pa_step_maps(const int32_t* cache_lens, const int32_t* new_lens, int B,
                                  const int32_t* free_blocks, int num_free,
                                  const int32_t* free_count, int32_t* block_tables, int max_blocks,
                                  int block_size, int num_blocks, int max_seq_len,
                                  int32_t* seq_lens, int32_t* q_start, int32_t* positions,
                                  int64_t* slots, int num_rows, int32_t* free_left,
                                  int* device_error, struct CUstream_st* stream) {
    if (!free_blocks || !free_count || !q_start || !free_left || (num_rows > 0 && (!positions || !slots)) ||
        (B != 0 && (!cache_lens || !new_lens || !block_tables || !seq_lens)))
        return PA_ERR_NULL;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (B < 0 || B > pa::kMaxBatch || max_blocks < 1 || num_blocks < 1 || max_seq_len < 1 ||
        num_free < 0 || num_rows < 0)
        return PA_ERR_SHAPE;
    if (static_cast<int64_t>(max_blocks) * block_size > INT32_MAX) return PA_ERR_SHAPE;
    auto off = [](const void* p, unsigned unit) { return (reinterpret_cast<uintptr_t>(p) & (unit - 1)) != 0; };
    if (off(cache_lens, 4) || off(new_lens, 4) || off(free_blocks, 4) || off(free_count, 4) ||
        off(block_tables, 4) || off(seq_lens, 4) || off(q_start, 4) || off(positions, 4) || off(slots, 8) ||
        off(free_left, 4) || off(device_error, 4))
        return PA_ERR_ALIGN;
    // (No requests: the rows are all padding, and are written as such, so that
    // no later call takes slots of the step before.)
    // Every block of the grid reads the inputs and block 0 writes these
    // outputs meanwhile: they must be other memory.
    const size_t nb = static_cast<size_t>(B) * 4;
    if (overlap(seq_lens, nb, cache_lens, nb) || overlap(seq_lens, nb, new_lens, nb) ||
        overlap(q_start, nb + 4, cache_lens, nb) || overlap(q_start, nb + 4, new_lens, nb) ||
        overlap(free_left, 4, free_count, 4))
        return PA_ERR_SHAPE;
    int* err = device_error;
    if (!err && pa::append_error_address(&err) != cudaSuccess) return PA_ERR_CUDA;
    pa::StepArgs a{};
    a.cache_lens = cache_lens;
    a.new_lens = new_lens;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.tables = block_tables;
    a.seq_lens = seq_lens;
    a.q_start = q_start;
    a.positions = positions;
    a.slots = slots;
    a.free_left = free_left;
    a.err = err;
    a.B = B;
    a.max_blocks = max_blocks;
    a.num_free = num_free;
    a.shift = block_size == 16 ? 4 : 5;
    a.num_blocks = num_blocks;
    a.limit = std::min(max_seq_len, max_blocks * block_size);
    a.T = num_rows;
    cudaLaunchConfig_t cfg = {};
    const int64_t want = (static_cast<int64_t>(num_rows) + pa::kStepThreads - 1) / pa::kStepThreads;
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, pa::kSms))));
    cfg.blockDim = dim3(pa::kStepThreads);
    cfg.dynamicSmemBytes = (2 * static_cast<size_t>(B) + 1) * 4;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    // Above the default limit, that of the largest batch: it belongs to the
    // function, which other threads launch with other batches.
    if (cfg.dynamicSmemBytes > 46 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void*>(pa::step_maps_kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (2 * pa::kMaxBatch + 1) * 4) != cudaSuccess)
        return PA_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pa::step_maps_kernel, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
