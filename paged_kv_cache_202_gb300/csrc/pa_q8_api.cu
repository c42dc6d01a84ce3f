// Attention over a paged cache held in 8 bits: argument checks, plans and launches
// of pa_decode_q8 and pa_prefill_q8.
#include <algorithm>
#include <cmath>

#include "pa.h"
#include "pa_internal.h"
#include "pa_plan.h"

namespace pa {
namespace {

// The pools' tensor maps, kept in the plan while the pools are the same.
bool pool_maps(pa_plan* plan, const void* k_pool, const void* v_pool, int rows, int D, int block_size) {
    const MapKey kk{k_pool, rows, D, block_size, 1}, vk{v_pool, rows, D, block_size, 1};
    if (!(plan->kkey == kk)) {
        plan->kkey = MapKey{};
        if (!encode_q8_map(&plan->kmap, k_pool, rows, D, block_size)) return false;
        plan->kkey = kk;
    }
    if (!(plan->vkey == vk)) {
        plan->vkey = MapKey{};
        if (!encode_q8_map(&plan->vmap, v_pool, rows, D, block_size)) return false;
        plan->vkey = vk;
    }
    return true;
}

// The split decode (pa_split_q8.cu) and its merge; q_start: T rows, a few queries a
// sequence, else one each.
pa_status decode_split(pa_plan* plan, const void* q, const int32_t* q_start, int T, int max_q, const void* k_pool, const void* v_pool, const float* k_scale,
                       const float* v_scale, const int32_t* tables, int max_blocks, const int32_t* seq_lens, int B,
                       int Hq, int Hkv, int D, int block_size, int num_blocks, int max_seq_len, float scale_log2,
                       void* out, int out_bf16, const SplitShape& sh, cudaStream_t stream) {
    SplitLaunch L{sh.kind, D, block_size, sh.NT, sh.warps, 0, sh.smem};
    L.mq = sh.mq;
    int per_sm = 0;
    for (const OccKey& o : plan->occ)
        if (o.kind == L.kind && o.D == D && o.BS == block_size && o.NT == L.NT && o.warps == L.warps && o.smem == L.smem && o.mq == L.mq)
            per_sm = o.blocks_per_sm;
    if (per_sm == 0) {
        cudaError_t e;
        per_sm = split_q8_blocks_per_sm(L, &e);
        if (e != cudaSuccess || per_sm < 1) return PA_ERR_CUDA;
        plan->occ.push_back(OccKey{L.kind, D, block_size, L.NT, L.warps, L.smem, per_sm, L.mq, 0, 0, 0});
    }
    const SplitGrid gr = split_grid(sh, B, D, block_size, static_cast<int64_t>(T) * Hq, plan->num_sms, per_sm);
    L.blocks = gr.blocks;
    const pa_status st = grow_workspace(plan, gr.workspace_bytes(), stream, true);
    if (st != PA_OK) return st;
    if (!pool_maps(plan, k_pool, v_pool, num_blocks * Hkv, D, block_size)) return PA_ERR_CUDA;
    char* const ws = static_cast<char*>(plan->ws);
    SplitQ8Args a{};
    a.q = static_cast<const uint16_t*>(q);
    a.tables = tables;
    a.seq_lens = seq_lens;
    a.out = out;
    a.ws_meta = reinterpret_cast<int*>(ws);
    a.ws_ml = reinterpret_cast<float*>(ws + gr.meta_bytes);
    a.ws_acc = reinterpret_cast<float*>(ws + gr.meta_bytes + gr.ml_bytes);
    a.err = plan->err;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.g = Hq / Hkv;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.max_seq_len = max_seq_len;
    a.scale_log2 = scale_log2;
    a.out_bf16 = out_bf16;
    set_split_plan(&a, sh, gr);
    a.probe_wait = wait_probe();
    a.q_start = q_start;
    a.nq = max_q;
    a.num_q = T;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    if (plan->ev_start) cudaEventRecord(plan->ev_start, stream);
    cudaError_t e = launch_split_q8(L, plan->kmap, plan->vmap, a, stream);
    if (plan->ev_stop) cudaEventRecord(plan->ev_stop, stream);
    if (e != cudaSuccess) return PA_ERR_CUDA;
    e = launch_merge_q8(a, D, L.mq, gr.ranges, stream);
    plan->last_path = PA_PATH_MMA;
    plan->last_blocks = L.blocks;
    plan->last_warps = gr.NW;
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The tcgen05 kernel (pa_prefill_q8.cu). Two tiles a block take in half the keys and
// values per row, and a block's two tiles take 1.5 to 1.6 times as long as one. So: one
// tile a block while its grid is at most one wave of blocks (those of few blocks cut
// the keys too), or when every sequence fits one; else two tiles. Measured, Hq 32,
// Hkv 8, one tile / two tiles: 1024 rows of 16384 tokens (256 blocks of one tile)
// 280 / 221 us, 1536 rows (384) 409 / 421, 2048 rows (512) 529 / 426; 1024-row prompts
// 35 / 28, 4096-row prompts 196 / 163; 16 sequences of 256 rows 341 / 268.
pa_status prefill(pa_plan* plan, const void* q, const int32_t* q_start, int T, int max_q, const void* k_pool,
                  const void* v_pool, const float* k_scale, const float* v_scale, const int32_t* tables,
                  int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int block_size, int num_blocks,
                  int max_seq_len, float scale_log2, void* out, int out_bf16, cudaStream_t stream) {
    const int64_t nq = std::min<int64_t>(max_q, T);
    const int qb = 128 / (Hq / Hkv);
    const int64_t blocks = (nq + qb - 1) / qb * static_cast<int64_t>(Hkv) * B;
    const int force = prefill_kernel_choice();  // a test may pin either build
    const bool pair = force == PA_PREFILL_AUTO ? nq > qb && blocks > plan->num_sms : force == PA_PREFILL_TWO_TILE;
    const int splits = pair ? 1 : prefill_split_count(B, Hq, Hkv, nq, max_seq_len, plan->num_sms);
    float* part = nullptr;
    if (splits > 1) {
        const size_t need = 64 + prefill_split_bytes(B, Hq, Hkv, nq, splits);
        const pa_status st = grow_workspace(plan, need, stream, true);
        if (st != PA_OK) return st;
        part = reinterpret_cast<float*>(static_cast<char*>(plan->ws) + 64);  // the first bytes: the splits' counters
    }
    if (!pool_maps(plan, k_pool, v_pool, num_blocks * Hkv, 128, block_size)) return PA_ERR_CUDA;
    if (plan->ev_start) cudaEventRecord(plan->ev_start, stream);
    const cudaError_t e = launch_prefill_q8(plan->kmap, plan->vmap, q, T, q_start, tables, seq_lens, k_scale, v_scale,
                                            out, plan->err, B, Hq, Hkv, max_blocks, num_blocks, max_seq_len, max_q,
                                            scale_log2, out_bf16, block_size, pair, part, splits, stream);
    if (plan->ev_stop) cudaEventRecord(plan->ev_stop, stream);
    plan->last_path = PA_PATH_PREFILL;
    plan->last_blocks = 0;
    plan->last_warps = 0;
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status attention_q8(const void* q, const int32_t* q_start, int T, int max_q, const void* k_pool,
                       const void* v_pool, const float* k_scale, const float* v_scale, const int32_t* tables,
                       int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int block_size,
                       int num_blocks, int max_seq_len, float scale, void* out, pa_dtype out_dtype,
                       pa_plan** plan_inout, cudaStream_t stream) try {
    if (!q || !k_pool || !v_pool || !k_scale || !v_scale || !tables || !seq_lens || !out || !plan_inout)
        return PA_ERR_NULL;
    if (out_dtype != PA_F32 && out_dtype != PA_BF16) return PA_ERR_DTYPE;
    if (block_size != 16 && block_size != 32) return PA_ERR_BLOCK_SIZE;
    if (B < 0 || B > kMaxBatch || T < 0 || max_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (D != 64 && D != 128) ||
        num_blocks < 1 || max_blocks < 1 || max_seq_len < 1 || !std::isfinite(scale) ||
        static_cast<int64_t>(num_blocks) * Hkv > INT32_MAX ||
        static_cast<int64_t>(max_blocks) * block_size > INT32_MAX || static_cast<int64_t>(T) * Hq > kMaxRows)
        return PA_ERR_SHAPE;
    if (q_start) {
        const int g = Hq / Hkv;
        if (D != 128 || g > 128 || 128 % g != 0 || max_blocks > 16384 || Hkv > kMaxGridYZ || !(scale > 0.f))
            return PA_ERR_SHAPE;
    }
    const uintptr_t vectors = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pool) |
                              reinterpret_cast<uintptr_t>(v_pool) | reinterpret_cast<uintptr_t>(out);
    const uintptr_t words = reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
                            reinterpret_cast<uintptr_t>(tables) | reinterpret_cast<uintptr_t>(seq_lens) |
                            reinterpret_cast<uintptr_t>(q_start);
    if ((vectors & 15u) || (words & 3u)) return PA_ERR_ALIGN;
    if (B == 0 || T == 0) return PA_OK;
    // All that depends on the arguments alone comes before the plan. A few queries a
    // sequence, up to 16 (query, head) columns a kv head, run on the decode's tiles: of
    // 64 sequences of 512 to 32768 tokens, 4 heads a kv head, 1 / 2 / 3 / 4 rows each take
    // 164 / 168 / 193 / 196 us there and 268 us on the tcgen05 kernel, whose tile of 128
    // rows is mostly empty; of 4 such sequences 18.5 / 18.7 / 25.1 / 25.5 and 25 us.
    const int64_t nq = q_start ? std::min<int64_t>(max_q, T) : 0;
    // (A page stream too long for those, by the call's bounds, leaves it to the tcgen05 kernel.)
    bool split = !q_start || (nq * (Hq / Hkv) <= 16 && prefill_kernel_choice() == PA_PREFILL_AUTO);
    SplitShape sh;
    split = split && split_shape(kSplitQ8, static_cast<int>(nq), B, Hq, Hkv, D, block_size, max_blocks, max_seq_len, &sh);
    if (!q_start && !split) return PA_ERR_SHAPE;
    const pa_status st = ensure_plan(plan_inout, stream, true);
    if (st != PA_OK) return st;
    pa_plan* const plan = *plan_inout;
    const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    if (split)
        return decode_split(plan, q, q_start, T, static_cast<int>(nq), k_pool, v_pool, k_scale, v_scale, tables,
                            max_blocks, seq_lens, B, Hq, Hkv, D, block_size, num_blocks, max_seq_len, scale_log2, out,
                            out_dtype == PA_BF16, sh, stream);
    return prefill(plan, q, q_start, T, max_q, k_pool, v_pool, k_scale, v_scale, tables, max_blocks, seq_lens, B, Hq,
                   Hkv, block_size, num_blocks, max_seq_len, scale_log2, out, out_dtype == PA_BF16, stream);
} catch (...) {  // host memory
    return PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

extern "C" {

pa_status pa_decode_q8(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
                       const float* v_scale, const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
                       int B, int Hq, int Hkv, int D, int block_size, int num_blocks, int max_seq_len, float scale,
                       void* out, pa_dtype out_dtype, pa_plan** plan_inout, struct CUstream_st* stream) {
    return pa::attention_q8(q, nullptr, B, 1, k_pool, v_pool, k_scale, v_scale, block_tables, max_blocks, seq_lens, B,
                            Hq, Hkv, D, block_size, num_blocks, max_seq_len, scale, out, out_dtype, plan_inout,
                            reinterpret_cast<cudaStream_t>(stream));
}

pa_status pa_prefill_q8(const void* q, const int32_t* q_start, int num_queries, int max_q, const void* k_pool,
                        const void* v_pool, const float* k_scale, const float* v_scale, const int32_t* block_tables,
                        int max_blocks, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int block_size,
                        int num_blocks, int max_seq_len, float scale, void* out, pa_dtype out_dtype,
                        pa_plan** plan_inout, struct CUstream_st* stream) {
    if (!q_start) return PA_ERR_NULL;
    return pa::attention_q8(q, q_start, num_queries, max_q, k_pool, v_pool, k_scale, v_scale, block_tables, max_blocks,
                            seq_lens, B, Hq, Hkv, D, block_size, num_blocks, max_seq_len, scale, out, out_dtype,
                            plan_inout, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
