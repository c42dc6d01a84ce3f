// Split paged decode over a cache held in 8 bits (pa_decode_q8): the page stream of
// pa_split.cuh, cut and merged as there, with a pipeline and a tile of its own.
//
// With kc, vc the codes and ks, vs the scales of a token's block,
//   s'_t = scale log2(e) ks (q . kc_t) + log2(vs),   w_t = 2^(s'_t - m),
//   O = sum w_t vc_t,   l = sum w_t / vs,   out = O / l:
// the values' scales sit in the exponents, so the value product takes the codes as
// they are, and its weights, rounded to f16, keep 11 bits relative to the largest
// for any mix of the scales that there are (pa_q8.cuh); l takes them unrounded. The
// output in bf16 is as near to exact arithmetic as one of 32-bit weights (1.67e-3 of its
// norm against 1.66e-3; in float32 1.4e-4 to 2.0e-4). The reference m is raised only
// when a score exceeds it by more than 8, so that most chunks need no maximum
// across the warp (any reference gives the same quotient); weights are taken times
// 2^7, so that f16 holds them up to there and down to 2^-32 of the largest. Codes become
// f16 exactly. A query head becomes f16 after a power of two brings its largest
// element to [2^8, 2^9), which keeps bf16's 8 bits down to 2^-26 of it.
//
// A warp takes a chunk of 32 tokens (64 at D = 64), 8 KB of codes, while the next
// one is on its way. S^T[16 tokens x 8 heads] = K Q^T and O^T[16 dims x 8 heads] +=
// V^T W^T run in m16n8k16 tiles. Both contractions' orders are free, so both
// operands come out of shared memory four neighbouring codes a thread, two of them
// the low half's pair of a fragment and two the high half's:
//   * keys: ldmatrix gives thread 4 r + c codes 4 c .. 4 c + 3 of 16 in row r; they are
//     k = 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of a k-step, and the query fragment holds the
//     same elements there;
//   * values: the bytewise transposing ldmatrix gives it rows 4 c .. 4 c + 3 of columns
//     r and r + 8; its row j is token j (j ^ 2 above 7) of the 16, and the keys' rows
//     are addressed so that row i of the scores is the token of k = i. That order also
//     puts the eight rows of every access in different banks.
//
// The scales and table entries of up to 32 pages (a batch) are read by a lane each,
// a batch ahead, and reach the tiles by shuffles.
#include <algorithm>

#include "pa_q8.cuh"
#include "pa_split.cuh"

namespace pa {
namespace split {

// Token of row i of a 16-row tile of the scores (see above).
__device__ __forceinline__ int q8_token(int i) {
    const int j = 4 * ((i & 7) >> 1) + (i & 1) + (i & 8 ? 2 : 0);
    return j < 8 ? j : j ^ 2;
}

// MQ: several queries per sequence (its newest tokens); column c of the tile is query
// c / g and head c % g, and query i sees the tokens before the last nqb - 1 - i.
template <int D, int NT, bool MQ>
struct Q8State {
    static constexpr bool kQS = NT == 2;           // query rows in a region of their own, reread at every chunk
    static constexpr int CT = kQ8ChunkBytes / (2 * D);
    static constexpr int KS = D / 16;              // k-steps of the scores, m-tiles of the values
    static constexpr int QP = mq_q_pitch(D);       // pitch of the query rows in the region
    static constexpr float kRaise = 8.f, kBias = 7.f;
    uint32_t qb[kQS ? 1 : KS][NT][2];              // Q^T fragments, held unless kQS
    float qs[NT][2];                               // the power of two of this thread's columns
    float o[KS][NT][4];
    float m[NT][2], l[NT][2];

    // Elements 16 kk + 4 c .. + 3 of query row `row`.
    static __device__ __forceinline__ uint32_t q_addr(uint32_t qst, int row, int lane, int kk) {
        return qst + row * QP + (16 * kk + 4 * (lane & 3)) * 2;
    }

    // Row of q and out of column c: g heads of each of the queries, Hq rows apart.
    static __device__ __forceinline__ int row_of(int c, int g, int Hq) { return MQ ? c / g * Hq + c % g : c; }

    // q: the segment's first query row, of nh; qst: the warp's region for them (kQS).
    __device__ __forceinline__ void start(const uint16_t* q, uint32_t qst, int nh, int lane, int g, int Hq) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + (lane >> 2);
            const uint16_t* const src = q + static_cast<size_t>(row_of(row, g, Hq)) * D + 4 * (lane & 3);
            uint2 w[KS];
            float a = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
                w[kk] = row < nh ? __ldg(reinterpret_cast<const uint2*>(src + 16 * kk)) : make_uint2(0, 0);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
                a = fmaxf(a, fmaxf(fmaxf(fabsf(bf16_lo(w[kk].x)), fabsf(bf16_hi(w[kk].x))),
                                   fmaxf(fabsf(bf16_lo(w[kk].y)), fabsf(bf16_hi(w[kk].y)))));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            // 2^(e - 8) for the largest's exponent e, at least 2^-126. (Infinities stay.)
            const uint32_t e = max(__float_as_uint(a) >> 23, 9u);
            const float s = __uint_as_float((e - 8u) << 23), inv = __uint_as_float((262u - e) << 23);
#pragma unroll
            for (int j = 0; j < 2; ++j) qs[nt][j] = __shfl_sync(0xffffffffu, s, 8 * (lane & 3) + 4 * j);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const uint32_t b0 = pack_f16x2(bf16_lo(w[kk].x) * inv, bf16_hi(w[kk].x) * inv);
                const uint32_t b1 = pack_f16x2(bf16_lo(w[kk].y) * inv, bf16_hi(w[kk].y) * inv);
                if constexpr (kQS) {
                    if (row < nh)
                        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(q_addr(qst, row, lane, kk)), "r"(b0), "r"(b1)
                                     : "memory");
                } else {
                    qb[kk][nt][0] = b0;
                    qb[kk][nt][1] = b1;
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = -INFINITY;
                l[nt][j] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
        }
        if constexpr (kQS) __syncwarp();
    }

    // The 16-byte chunk `c` of row `tok` of a page stack with the swizzle of its rows' width.
    static __device__ __forceinline__ uint32_t at(uint32_t region, int c, int tok) {
        return D == 128 ? region + tok * 128 + ((c ^ (tok & 7)) << 4) : region + tok * 64 + ((c ^ ((tok >> 1) & 3)) << 4);
    }

    // The chunk's nv tokens, of rem before the sequence's end (MQ). Lane pg0 + j holds page j's scales: the keys' times the
    // score scale and log2 e (ksl), and log2 of the values' (lvs). far: value scales far apart
    // (pa_q8.cuh).
    template <int BS>
    __device__ __forceinline__ void chunk(uint32_t kst, uint32_t vst, int nv, int lane, int pg0, float ksl, float lvs,
                                          uint32_t qst, int nh, int rem, int nqb, int g, bool far) {
        if (nv < CT) {
            // Behind the end: whatever is there. No value of it may be NaN.
            for (int i = lane; i < (CT - nv) * (D / 16); i += 32)
                st_shared_v4(vst + nv * D + i * 16, make_uint4(0, 0, 0, 0));
            __syncwarp();
        }
#pragma unroll 1
        for (int sub = 0; sub < CT; sub += 32) {
            const int left = nv - sub;  // tokens before the end
            if (CT > 32 && left <= 0) break;
            float s[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][nt][i] = 0.f;
            const int krow = sub + q8_token(lane & 15);
#pragma unroll
            for (int k2 = 0; k2 < KS / 2; ++k2) {
                uint32_t b[2][NT][2];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (kQS) {
                            const int row = nt * 8 + (lane >> 2);
                            const uint2 w = row < nh ? lds_u64(q_addr(qst, row, lane, 2 * k2 + kk)) : make_uint2(0, 0);
                            b[kk][nt][0] = w.x;
                            b[kk][nt][1] = w.y;
                        } else {
                            b[kk][nt][0] = qb[2 * k2 + kk][nt][0];
                            b[kk][nt][1] = qb[2 * k2 + kk][nt][1];
                        }
                    }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t r[4];
                    ldsm_x4(at(kst, 2 * k2 + (lane >> 4), krow + 16 * t), r[0], r[1], r[2], r[3]);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const uint32_t a0 = q8::to_f16x2(r[2 * kk]), a1 = q8::to_f16x2(r[2 * kk + 1]);
                        const uint32_t a2 = q8::hi_to_f16x2(r[2 * kk]), a3 = q8::hi_to_f16x2(r[2 * kk + 1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(s[t][nt], a0, a1, a2, a3, b[kk][nt][0], b[kk][nt][1]);
                    }
                }
            }
            // To the log2 domain; the end masked.
            float inv[2];  // 2^24 / vs
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int pg = pg0 + (sub + t * 16) / BS;
                const float ks = __shfl_sync(0xffffffffu, ksl, pg), lv = __shfl_sync(0xffffffffu, lvs, pg);
                inv[t] = fast_exp2(q8::kSumBias - lv);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[t][nt][i] = fmaf(s[t][nt][i], ks * qs[nt][i & 1], lv);
            }
            if ((MQ ? min(left, rem - sub - (nqb - 1)) : left) < 32) {
                const int ta = q8_token(lane >> 2), tb = q8_token((lane >> 2) + 8);
                int lim[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        lim[nt][j] = MQ ? min(left, rem - sub - (nqb - 1 - (nt * 8 + 2 * (lane & 3) + j) / g)) : left;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (16 * t + (i >= 2 ? tb : ta) >= lim[nt][i & 1]) s[t][nt][i] = -INFINITY;
            }
            float mx[NT][2];
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[nt][j] = fmaxf(max3(s[0][nt][j], s[0][nt][2 + j], s[1][nt][j]), s[1][nt][2 + j]);
                    raise |= mx[nt][j] > m[nt][j] + kRaise;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = mx[nt][j];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        if (x > m[nt][j] + kRaise) {
                            const float f = fast_exp2(m[nt][j] - x);  // 0 at the segment's first tokens
                            l[nt][j] = q8::times_exp2(l[nt][j], m[nt][j] - x);
                            m[nt][j] = x;
#pragma unroll
                            for (int mt = 0; mt < KS; ++mt) {
                                o[mt][nt][j] *= f;
                                o[mt][nt][2 + j] *= f;
                            }
                        }
                    }
            }
            uint32_t pb[2][NT][2];  // W^T fragments: [tile][n-tile][token half]
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float base[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) base[j] = (m[nt][j] == -INFINITY ? 0.f : m[nt][j]) - kBias;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = fast_exp2(s[t][nt][i] - base[i & 1]);
                    pb[t][nt][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
                    pb[t][nt][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
                    float e = inv[t];
                    if (far) {  // once more, without the value scale
                        e = 1.f;
                        const float lv = __shfl_sync(0xffffffffu, lvs, pg0 + (sub + t * 16) / BS) - q8::kSumBias;
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = fast_exp2(s[t][nt][i] - base[i & 1] - lv);
                    }
                    l[nt][0] = fmaf(p[0] + p[2], e, l[nt][0]);
                    l[nt][1] = fmaf(p[1] + p[3], e, l[nt][1]);
                }
            }
            // Rows of the value tiles: token j, or j ^ 2, of the 16.
            const int vrow = sub + ((lane & 8) ? (lane & 15) ^ 2 : lane & 15);
#pragma unroll
            for (int m2 = 0; m2 < KS / 2; ++m2)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t r[4];
                    ldsm_b8_trans_x2(at(vst, 2 * m2 + (lane >> 4), vrow + 16 * t), r[0], r[1], r[2], r[3]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = q8::to_f16x2(r[2 * h]), a1 = q8::to_f16x2(r[2 * h + 1]);
                        const uint32_t a2 = q8::hi_to_f16x2(r[2 * h]), a3 = q8::hi_to_f16x2(r[2 * h + 1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16_16816(o[2 * m2 + h][nt], a0, a1, a2, a3, pb[t][nt][0], pb[t][nt][1]);
                    }
                }
        }
    }

    __device__ __forceinline__ void finish(const SplitArgs& a, uint32_t row0, int nh, bool full, bool poison, int slot,
                                           int lane) {
        const int dr = lane >> 2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float lt = l[nt][j];
                lt += __shfl_xor_sync(0xffffffffu, lt, 4);
                lt += __shfl_xor_sync(0xffffffffu, lt, 8);
                lt += __shfl_xor_sync(0xffffffffu, lt, 16);
                const int head = nt * 8 + 2 * (lane & 3) + j;
                if (head >= nh) continue;
                const float f = full ? q8::kSumFactor / lt : 1.f;
                const size_t part = static_cast<size_t>(slot) * a.GS + head, row = row0 + row_of(head, a.g, a.Hq);
#pragma unroll
                for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int d = mt * 16 + dr + 8 * r;
                        const float v = poison ? 0.f : o[mt][nt][2 * r + j] * f;
                        if (!full) a.ws_acc[part * D + d] = v;
                        else if (a.out_bf16) static_cast<uint16_t*>(a.out)[row * D + d] = f32_to_bf16_bits(v);
                        else static_cast<float*>(a.out)[row * D + d] = v;
                    }
                if (!full && dr == 0) {
                    a.ws_ml[part * 2] = poison ? __int_as_float(0x7fc00000) : m[nt][j];
                    a.ws_ml[part * 2 + 1] = poison ? 0.f : lt;
                }
            }
        }
    }
};

// A batch: up to 32 consecutive pages of one segment within one range.
struct Q8Batch {
    int b, u, p, cnt;   // sequence, kv unit, first page, pages
    int id;             // range
    int start, end;     // whether it holds the range's first (last) pages of the segment
    int pad;
};

template <int D, int BS, int NT, bool MQ>
__device__ __forceinline__ void q8_body(const CUtensorMap* kmap, const CUtensorMap* vmap, const SplitQ8Args& a) {
    using State = Q8State<D, NT, MQ>;
    constexpr int CP = State::CT / BS;                 // pages per chunk
    constexpr uint32_t kHalf = kQ8ChunkBytes / 2;      // K, or V, of a chunk
    constexpr int S = kQ8Stages;
    static_assert(S == 2 && CP >= 1 && CP <= 4, "stages");
    extern __shared__ uint8_t smem_raw[];
    const int lane = threadIdx.x & 31, W = blockDim.x >> 5;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    int* pre = reinterpret_cast<int*>(smem_raw + (base - raw));
    int* len = pre + (a.B + 1);
    const uint32_t ring = base + a.lens_bytes + static_cast<uint32_t>(warp * S) * kQ8ChunkBytes;
    const uint32_t after = base + a.lens_bytes + static_cast<uint32_t>(W * S) * kQ8ChunkBytes;
    const uint32_t rec = after + warp * kQ8RecordBytes;                       // four batches
    const uint32_t bars = after + W * kQ8RecordBytes + warp * S * 8;
    const uint32_t probe_bar = after + W * (kQ8RecordBytes + S * 8);          // nothing completes it
    const uint32_t my_q = probe_bar + 16 + static_cast<uint32_t>(warp * a.q_bytes);

    if (threadIdx.x == 0) {
        prefetch_tensormap(kmap);
        prefetch_tensormap(vmap);
        mbar_init(probe_bar, 1);
        fence_barrier_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    scan_lengths<BS, false, MQ>(a.seq_lens, a.B, min(a.max_seq_len, a.max_blocks * BS), pre, len, a.err,
                                MQ ? a.q_start : nullptr, a.nq, a.num_q);

    const int P = a.U * pre[a.B];
    const int NW = gridDim.x * W;
    const Q8Groups cut(P, NW, CP, a.GS);
    const int per = cut.at[3], groups = (P + per - 1) / per;
    const int nd = cut.cut() ? 2 * groups : 0;
    if (blockIdx.x == 0) {  // for the merge
        for (int i = threadIdx.x; i <= a.B; i += blockDim.x) a.ws_meta[kMetaHeader + i] = pre[i];
        if (threadIdx.x == 0) {
            a.ws_meta[0] = P;
            a.ws_meta[1] = per;
            a.ws_meta[2] = NW;
            a.ws_meta[4] = cut.at[1];
            a.ws_meta[5] = cut.at[2];
        }
    }
    const int gw = warp * gridDim.x + blockIdx.x;  // few groups: spread over the SMs
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();

    // ---- the batches of this warp's ranges, one after the other
    auto part = [&](int i, int k) {  // (shorter, or empty, at the stream's end)
        const int first = k == 0 ? 0 : k == 1 ? cut.at[1] : cut.at[2];
        const int last = k == 0 ? cut.at[1] : k == 1 ? cut.at[2] : per;
        return Range{i * per + first, min(i * per + last, P), nd > 0 ? 3 * i + k : i};
    };
    Range ri = gw < groups ? part(gw, 0) : Range{0, 0, -1};
    int claimed = 0;  // lane 0: the next dynamic range, asked for a chunk before it is looked at
    bool asked = false;
    auto ask = [&] {
        if (nd > 0 && lane == 0) claimed = atomicAdd(a.ws_meta + 3, 1);
        asked = true;
    };
    auto answer = [&] {
        while (true) {
            const int j = nd > 0 ? __shfl_sync(0xffffffffu, claimed, 0) : 0;
            asked = false;
            ri = Range{0, 0, -1};
            if (j >= nd) return;
            ri = part(j % groups, 1 + j / groups);
            if (ri.x0 < ri.x1) return;
            ask();
        }
    };
    Cursor g{0, 0, 0, 0};
    auto locate = [&](int x) {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.U * pre[mid] <= x) lo = mid; else hi = mid - 1;
        }
        const int nb = seq_pages(pre, lo), off = x - a.U * pre[lo], u = off / nb;
        return Cursor{lo, u, off - u * nb, nb};
    };
    if (ri.id < 0) {
        ask();
        answer();
        if (ri.id < 0) return;
    }
    int xg = ri.x0, made = 0;
    g = locate(xg);
    int n_cnt = 0, n_kvh = 0, n_tbl = -1;  // the batch ahead: pages, kv head, lane j's table entry
    auto make_batch = [&] {
        if (xg == ri.x1) {
            if (ri.id >= 0) {
                if (!asked) ask();
                answer();
                if (ri.id >= 0) {
                    xg = ri.x0;
                    g = locate(xg);
                }
            }
            if (ri.id < 0) {
                n_cnt = 0;
                return;
            }
        }
        n_cnt = min(min(32, g.nb - g.p), ri.x1 - xg);
        n_kvh = g.u / a.nslices;
        n_tbl = lane < n_cnt ? __ldg(a.tables + static_cast<size_t>(g.b) * a.max_blocks + g.p + lane) : -1;
        if (lane == 0) {
            const uint32_t r = rec + (made & 3) * sizeof(Q8Batch);
            sts_v4i(r, g.b, g.u, g.p);
            asm volatile("st.shared.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(r + 16), "r"(ri.id),
                         "r"(xg == ri.x0 || g.p == 0 ? 1 : 0), "r"(g.p + n_cnt == g.nb || xg + n_cnt == ri.x1 ? 1 : 0),
                         "r"(n_cnt)
                         : "memory");
        }
        if (xg == ri.x0 || g.p == 0) {  // the segment's query rows, towards the time its first chunk is here
            const int first = MQ ? a.q_start[g.b] : g.b, slice = g.u - n_kvh * a.nslices;
            const int rows = MQ ? a.q_start[g.b + 1] - first : 1, heads = min(a.GS, a.g - slice * a.GS);
            const int64_t row = static_cast<int64_t>(first) * a.Hq + n_kvh * a.g + slice * a.GS;
            for (int i = lane * 64; i < rows * heads * D; i += 32 * 64) {
                const int r = i / (heads * D);
                prefetch_l1(a.q + (row + static_cast<int64_t>(r) * a.Hq) * D + (i - r * heads * D));
            }
        }
        ++made;
        xg += n_cnt;
        g.p += n_cnt;
        if (g.p == g.nb) {
            g.p = 0;
            if (++g.u == a.U) {
                g.u = 0;
                do {
                    ++g.b;
                } while (g.b < a.B && seq_pages(pre, g.b) == 0);
                g.nb = g.b < a.B ? seq_pages(pre, g.b) : 0;
            }
        }
        __syncwarp();
    };
    // ---- the batch whose pages are being copied
    const uint32_t one = elect_one();
    int cnt = 0, next = 0, kvh = 0, tbl = -1;
    uint32_t bad = 0, badstage = 0, phase = 0;  // (badstage: two stages' bits, then value scales seen, see work_on)
    float ks = 1.f, vs = 1.f;
    bool issue_done = false;
    auto open = [&] {  // false: there is none
        if (n_cnt == 0) return false;
        cnt = n_cnt;
        next = 0;
        kvh = n_kvh;
        tbl = n_tbl;
        const bool out = lane < cnt && (tbl < 0 || tbl >= a.num_blocks);
        bad = __ballot_sync(0xffffffffu, out);
        if (bad && lane == 0) atomicOr(a.err, kErrTable);
        ks = vs = 1.f;
        if (lane < cnt && !out) {
            const size_t at = static_cast<size_t>(tbl) * a.Hkv + kvh;
            ks = a.k_scale[at];
            vs = a.v_scale[at];
        }
        return true;
    };
    auto issue = [&](int s) {
        if (next == cnt && !open()) {
            issue_done = true;
            return;
        }
        const int n = min(CP, cnt - next);
        const uint32_t bar = bars + 8 * s, stg = ring + s * kQ8ChunkBytes;
        const bool skip = (bad >> next) & ((1u << n) - 1u);
        badstage = skip ? badstage | (1u << s) : badstage & ~(1u << s);
        if (one) mbar_arrive_expect_tx(bar, skip ? 0u : n * (2u * BS * D));
        __syncwarp();
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            const int row = __shfl_sync(0xffffffffu, tbl, (next + j) & 31) * a.Hkv + kvh;
            const uint32_t on = j < n && !skip ? one : 0u;
            tma_load_3d_if(on, stg + j * (BS * D), kmap, 0, 0, row, bar);
            tma_load_3d_if(on, stg + kHalf + j * (BS * D), vmap, 0, 0, row, bar);
        }
        next += n;
        // The batch ahead: its table entries are on their way while this one's last
        // chunk is waited for. A dynamic piece is claimed late, so that the pieces go
        // to whichever warp is ahead.
        if (next + CP >= cnt && xg == ri.x1 && ri.id >= 0 && !asked) ask();
        if (next == cnt) make_batch();
    };
    // ---- the batch whose pages are being worked on
    State st;
    float ksl = 1.f, lvs = 0.f;
    int opened = 0, cb = 0, cu = 0, cp = 0, ccnt = 0, ci = 0, id = 0, end = 0;
    int p_first = 0, nh = 0, nqb = 1;
    uint32_t row0 = 0;
    bool poison = false;
    auto work_on = [&](float ks, float vs) {  // the next batch, with the scales of its pages
        const uint32_t r = rec + (opened & 3) * sizeof(Q8Batch);
        const int4 x = lds_v4i(r), y = lds_v4i(r + 16);
        ++opened;
        cb = x.x;
        cu = x.y;
        cp = x.z;
        id = y.x;
        end = y.z;
        ccnt = y.w;
        ci = 0;
        if (y.y) {
            const int h = cu / a.nslices, slice = cu - h * a.nslices;
            if constexpr (MQ) {
                const int first = a.q_start[cb];
                nqb = a.q_start[cb + 1] - first;
                nh = nqb * a.g;
                row0 = static_cast<uint32_t>(first) * a.Hq + h * a.g;
            } else {
                nh = min(a.GS, a.g - slice * a.GS);
                row0 = static_cast<uint32_t>(cb) * a.Hq + h * a.g + slice * a.GS;
            }
            st.start(a.q + static_cast<size_t>(row0) * D, my_q, nh, lane, a.g, a.Hq);
            p_first = cp;
            poison = false;
        }
        ksl = ks * a.scale_log2;
        lvs = q8::log2_of(vs, ks);
        // The value scales' range so far as a bit for every 2^6.17 (from 2^-65: the logarithm is an
        // approximation), behind the stages' bits: one reduction, and no register of its own (the
        // kernels of two n-tiles have none left).
        const uint32_t now = __reduce_or_sync(0xffffffffu, lane < ccnt ? 4u << ((__float2int_rd(lvs) + 65) * 83 >> 9) : 0u);
        badstage = (y.y ? badstage & 3u : badstage) | now;
    };
    make_batch();
    issue(0);
    {
        const float k0 = ks, v0 = vs;  // a second chunk may be of the next batch
        issue(1);
        work_on(k0, v0);
    }
    int s = 0;
    bool first = true;
    int in_flight = issue_done ? 1 : 2;
    while (true) {
        const uint32_t bar = bars + 8 * s, stg = ring + s * kQ8ChunkBytes;
        const bool ready = a.probe_wait && first ? mbar_wait_bounded(probe_bar, 0, kProbeLimitNs)
                                                 : mbar_wait_bounded(bar, (phase >> s) & 1u, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, ready)) {
            // Give up: report, wait (bounded) for this warp's copies in flight, return.
            if (lane == 0) atomicOr(a.err, kErrTimeout);
            for (int j = 0; j < in_flight; ++j)
                mbar_wait_bounded(bars + 8 * (s ^ j), (phase >> (s ^ j)) & 1u, kWaitLimitNs);
            return;
        }
        first = false;
        phase ^= 1u << s;
        const int n = min(CP, ccnt - ci);
        if ((badstage >> s) & 1u) {
            poison = true;
        } else {
            const int rem = len[cb] - (cp + ci) * BS;
            const uint32_t seen = badstage & ~3u;
            constexpr int kSteps = static_cast<int>(q8::kFarApart) * 83 / 512 - 1;  // so many lie within kFarApart
            st.template chunk<BS>(stg, stg + kHalf, min(n * BS, rem), lane, ci, ksl, lvs, my_q, nh, rem, nqb, a.g,
                                  31 - __clz(seen) - (__ffs(seen) - 1) > kSteps);
        }
        ci += n;
        __syncwarp();
        if (ci == ccnt && end) {
            const bool full = p_first == 0 && cp + ccnt == seq_pages(pre, cb);
            st.finish(a, row0, nh, full, poison, id * 2 + (p_first > 0 ? 0 : 1), lane);
        }
        if (ci == ccnt && in_flight == 2) work_on(ks, vs);  // the other stage holds its first chunk
        if (!issue_done) {
            fence_proxy_async_smem();
            issue(s);
        }
        if (issue_done && --in_flight == 0) break;
        s ^= 1;
    }
}

// One block an SM, of as many warps as 170 registers a thread and the shared memory
// allow: twelve, or eleven with two n-tiles.
//
// Measured (device time, split and merge; the copy rate is 6.8 TB/s). 64 sequences of
// 512 to 32768 tokens, 32 / 8 heads of 128: 132 us for 0.80 GB, 6.05 TB/s (0.89), the
// split kernel alone 124.8 us under the profiler with DRAM at 82 %; a kernel that only
// reads as many 2 KB pages takes 122 us, this one from L2 95 us, so DRAM bounds it,
// then the merge (7.4 us). 24 sequences of 8192 to 131072 tokens, 128 / 8 heads: 311 to
// 317 us for 1.95 GB, 6.2 TB/s (0.91); with two n-tiles the tiles take 274 us from L2. 32
// of 128 to 2048, 32 / 32 heads: 36.6 us, 4.4 TB/s: 5 us of start, uneven ends, the merge.
// One of 8191: 12.6 us: the chain of scan, table, scales and pages, and the merge.
// 64 sequences, 4 newest queries each: 193 to 199 us. Heads of 64, whose pages are 1 KB:
// 80 us for the first of these (0.73), 168 the second (0.85), 28.4 the third, 10.5 the
// fourth.
// Slower: one stage of 16 KB a warp (139 us for the first of these), smaller pieces
// at the end of the page stream (their partials cost the merge more than they even out).
template <int D, int BS, int NT, bool MQ>
__global__ void __launch_bounds__(32 * kQsMaxWarps, 1)
    q8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const SplitQ8Args a) {
    q8_body<D, BS, NT, MQ>(&kmap, &vmap, a);
}

constexpr int kMergeWarps = 16;  // of a block of the merge, at most

// The merge of the partials of a segment that was cut: one block per segment, `wpc`
// warps a column, each folding batches of eight neighbouring partials against a
// running maximum, then joined through shared memory (m = max m_i, l = sum l_i
// 2^(m_i - m), o = sum O_i 2^(m_i - m) / l). A segment's bounds are found once for all
// its columns, and a batch's loads are all in flight together.
__device__ __forceinline__ void ld_f(float (&v)[4], const float* p) {
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_f(float (&v)[2], const float* p) {
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p) : "memory");
}

template <int D, bool MQ>
__global__ void __launch_bounds__(32 * kMergeWarps, 1) q8_merge_kernel(const SplitQ8Args a, int wpc, int blocks) {
    constexpr int E = D / 32;  // elements a lane
    constexpr int kBatch = 8;
    __shared__ float sm_acc[kMergeWarps][D], sm_m[kMergeWarps], sm_l[kMergeWarps];
    __shared__ int sm_bad[kMergeWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Segment, and this block's share of its columns.
    const int seg = blockIdx.x / blocks, b = seg / a.U, u = seg - b * a.U;
    const int W = blockDim.x >> 5, col0 = (blockIdx.x - seg * blocks) * (W / wpc);
    const int col = col0 + warp / wpc, w = warp % wpc;
    griddep_wait();
    const int* pre = a.ws_meta + kMetaHeader;
    const int p0 = pre[b], nb = pre[b + 1] - p0;
    const int per = a.ws_meta[1], at1 = a.ws_meta[4], at2 = a.ws_meta[5];
    if (blockIdx.x == 0 && threadIdx.x == 0) a.ws_meta[3] = 0;  // dynamic-range counter, for the next call
    const int h = u / a.nslices, slice = u - h * a.nslices;
    auto put = [&](size_t row, const float (&v)[E]) {
        const size_t o = row * D + lane * E;
        if (a.out_bf16) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o);
            if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            else *dst = pack_bf16x2(v[0], v[1]);
        } else {
            float* dst = static_cast<float*>(a.out) + o;
            if constexpr (E == 4) *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            else *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[1]);
        }
    };
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    if (nb == 0) {  // an invalid sequence's rows are zeros (MQ: those that lie in the array)
        const int q0 = MQ ? max(a.q_start[b], 0) : b, q1 = MQ ? min(a.q_start[b + 1], a.num_q) : b + 1;
        const int heads = MQ ? a.g : min(a.GS, a.g - slice * a.GS);
        const int64_t rows = static_cast<int64_t>(max(q1 - q0, 0)) * heads;
        for (int64_t i = col0 == 0 ? warp : rows; i < rows; i += W)
            put((static_cast<size_t>(q0) + i / heads) * a.Hq + h * a.g + slice * a.GS + i % heads, acc);
        return;
    }
    const int sb = a.U * p0 + u * nb;
    auto range_of = [&](int x) {
        const int i = x / per, y = x - i * per;
        return at1 < per ? 3 * i + (y < at1 ? 0 : y < at2 ? 1 : 2) : i;
    };
    const int rf = range_of(sb), np = range_of(sb + nb - 1) - rf + 1;
    if (np == 1) return;  // finished inside one range by the split kernel
    const int nh = MQ ? (a.q_start[b + 1] - a.q_start[b]) * a.g : min(a.GS, a.g - slice * a.GS);
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    if (col < nh) {
        for (int i0 = w * kBatch; i0 < np; i0 += wpc * kBatch) {
            // The segment's first range left its partial in the tail slot, the others in the head's.
            auto part = [&](int i) { return (static_cast<size_t>(2 * (rf + i) + (i == 0 ? 1 : 0)) * a.GS + col); };
            const int n = min(kBatch, np - i0);
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) ml = *reinterpret_cast<const float2*>(a.ws_ml + part(i0 + lane) * 2);
            // (Past the last partial that one again, times 0. In one order, all before any use.)
            float v[kBatch][E];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) ld_f(v[k], a.ws_acc + part(min(i0 + k, np - 1)) * D + lane * E);
            bad |= __any_sync(0xffffffffu, ml.x != ml.x);  // the marker of a bad table entry
            float mb = ml.x;
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, off));
            mb = fmaxf(m, __shfl_sync(0xffffffffu, mb, 0));
            // No score that is a number: the sums, 0 or NaN, tell.
            const float base = mb == -INFINITY ? 0.f : mb, fo = fast_exp2(m - base), f = fast_exp2(ml.x - base);
            l = mb == -INFINITY ? l : q8::times_exp2(l, m - base);
            float lb = ml.x == -INFINITY ? ml.y : q8::times_exp2(ml.y, ml.x - base);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) lb += __shfl_xor_sync(0xffffffffu, lb, off);
            l += __shfl_sync(0xffffffffu, lb, 0);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] *= fo;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] = fmaf(v[k][i], fk, acc[i]);
            }
            m = mb;
        }
    }
    if (wpc > 1) {
        if (lane == 0) {
            sm_m[warp] = m;
            sm_l[warp] = l;
            sm_bad[warp] = bad;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) sm_acc[warp][lane * E + i] = acc[i];
        __syncthreads();
        if (w != 0 || col >= nh) return;
        float mt = -INFINITY;
        for (int i = 0; i < wpc; ++i) {
            mt = fmaxf(mt, sm_m[warp + i]);
            bad |= sm_bad[warp + i] != 0;
        }
        const float base = mt == -INFINITY ? 0.f : mt;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.f;
        for (int j = 0; j < wpc; ++j) {
            const float mj = sm_m[warp + j], f = fast_exp2(mj - base);
            l += mj == -INFINITY ? sm_l[warp + j] : q8::times_exp2(sm_l[warp + j], mj - base);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] = fmaf(sm_acc[warp + j][lane * E + i], f, acc[i]);
        }
    }
    if (col >= nh) return;
    const float inv = q8::kSumFactor / l;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = bad ? 0.f : acc[i] * inv;
    const size_t row0 = MQ ? static_cast<size_t>(a.q_start[b]) * a.Hq + h * a.g
                           : static_cast<size_t>(b) * a.Hq + h * a.g + slice * a.GS;
    put(row0 + (MQ ? static_cast<size_t>(col / a.g) * a.Hq + col % a.g : col), acc);
}

using Q8Fn = void (*)(CUtensorMap, CUtensorMap, SplitQ8Args);

Q8Fn select_q8(const SplitLaunch& L) {
    if (L.kind != kSplitQ8 || (L.NT != 1 && L.NT != 2)) return nullptr;
    const bool one = L.NT == 1;
    if (L.mq) {
        if (L.D != 128) return nullptr;
        if (L.BS == 16) return one ? q8_kernel<128, 16, 1, true> : q8_kernel<128, 16, 2, true>;
        return one ? q8_kernel<128, 32, 1, true> : q8_kernel<128, 32, 2, true>;
    }
    if (L.D == 128 && L.BS == 16) return one ? q8_kernel<128, 16, 1, false> : q8_kernel<128, 16, 2, false>;
    if (L.D == 128 && L.BS == 32) return one ? q8_kernel<128, 32, 1, false> : q8_kernel<128, 32, 2, false>;
    if (L.D == 64 && L.BS == 16) return one ? q8_kernel<64, 16, 1, false> : q8_kernel<64, 16, 2, false>;
    if (L.D == 64 && L.BS == 32) return one ? q8_kernel<64, 32, 1, false> : q8_kernel<64, 32, 2, false>;
    return nullptr;
}

}  // namespace split

int split_q8_blocks_per_sm(const SplitLaunch& L, cudaError_t* status) {
    split::Q8Fn fn = split::select_q8(L);
    int n = 0;
    // For every call in the process, whatever its size (as in pa_split.cu).
    *status = fn ? cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kScanSmemLimit))
                 : cudaErrorInvalidValue;
    if (*status == cudaSuccess)
        *status = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(fn), L.warps * 32,
                                                                L.smem);
    return *status == cudaSuccess ? n : 0;
}

// Warps a column: one for a batch of eight partials of the average segment; columns a
// block what that leaves of kMergeWarps. Measured (split and merge): a warp for eight
// against one for four, 64 sequences of 512 to 32768 tokens 132.5 / 134.3 us, 24 of 8192 to
// 131072 with 16 columns 313 / 322; against one for sixteen, 64 sequences 164 / 169 us, four
// 18.9 / 20.6.
cudaError_t launch_merge_q8(const SplitQ8Args& a, int D, int mq, int64_t ranges, cudaStream_t stream) {
    const int64_t units = static_cast<int64_t>(a.B) * a.U;
    int wpc = 1;
    const int64_t parts = ranges / units + 2;
    while (wpc < split::kMergeWarps && 8 * wpc < parts) wpc *= 2;
    const int cols = std::min(a.GS, split::kMergeWarps / wpc), blocks = (a.GS + cols - 1) / cols;
    if (units * blocks > INT32_MAX) return cudaErrorInvalidValue;
    auto fn = mq ? split::q8_merge_kernel<128, true>
                 : D == 128 ? split::q8_merge_kernel<128, false> : split::q8_merge_kernel<64, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * cols * wpc));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, a, wpc, blocks);
}

cudaError_t launch_split_q8(const SplitLaunch& L, const CUtensorMap& kmap, const CUtensorMap& vmap,
                            const SplitQ8Args& a, cudaStream_t stream) {
    split::Q8Fn fn = split::select_q8(L);
    if (!fn) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.blocks);
    cfg.blockDim = dim3(L.warps * 32);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, a);
}

}  // namespace pa
