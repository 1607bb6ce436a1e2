// rc_paged_scores_tc.cu -- the attention weight of each cached token, for many
// query rows, on the tensor cores (tcgen05).
//
// Transposed: S^T = K Q^T, so a thread holds one cached token's scores (a lane of
// TMEM) and its sum over the queries runs in one register, in one order; no two
// threads add to one entry.  A block has a range of the cached tokens of one
// (sequence, KV head) and goes over the head's query rows in blocks of up to
// 384, which stay in shared memory as three tiles while the cached tokens stream
// past, in pairs of tiles of 128:
//   warps 0, 1     issue the products of the pairs with an even, an odd number
//                  (one lane each); warp 0 owns TMEM: four places of 128 x 128
//                  scores, one for each tile of two pairs
//   warps 4 .. 19  four groups, one a place: exp2(S c - lse) and the sum over the
//                  columns, a token a thread.  One warp's chain of load, product
//                  sum, exponential and add leaves the units idle most of the
//                  time, so each scheduler has four of them (with two it took
//                  111 us for 757 x 5,788 tokens x 48 heads).  They also bring
//                  the query rows.
//   warps 20 .. 27 read K's codes from the pages (a pair of tiles ahead, in
//                  registers) and make them bf16 operand tiles, four warps for
//                  each tile of a pair
// With the queries kept, K is read and converted once per 384 rows, and the
// queries once per block: keeping K instead would read them for every 128
// tokens (430 MB of cache traffic for 757 x 5,788 tokens x 48 heads).
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

// 896 threads launched with 72 registers each; the warpgroups share them
// 40 + 4 x 80 + 2 x 72.
constexpr int kStThreads = 896;
constexpr int kStSums = 512;  // threads of the four groups
constexpr int kStTile = 128;
constexpr int kStQTiles = 3;  // query tiles in shared memory

enum : int {
    S_K_FULL = 0,    // [4] buffer 2 (pair & 1) + tile of the pair: K tile converted
    S_K_EMPTY = 4,   // [4] its products have finished
    S_S_FULL = 8,    // [4] scores of the K tile and a query tile in TMEM
    S_S_FREE = 12,   // [4] the group has read them
    S_Q_FULL = 16,   // the block's query rows are in place
    S_Q_EMPTY = 17,  // every group has the scores of the block before
    S_DRAIN = 18,
    S_COUNT = 19
};

template <int D>
struct StLayout {
    static constexpr uint32_t kTile = kStTile * D * 2;
    static constexpr uint32_t kK = 0;                          // [4]
    static constexpr uint32_t kQ = 4 * kTile;                  // [3]
    static constexpr uint32_t kMinus = kQ + kStQTiles * kTile;  // fp32 [3][128]: -lse log2(e)
    static constexpr uint32_t kBar = kMinus + kStQTiles * kStTile * 4;
    static constexpr uint32_t kMisc = kBar + 8 * S_COUNT;
    static constexpr uint32_t kTotal = kMisc + 16;
    static constexpr uint32_t kAlloc = kTotal + 1024;
};

// What a block does, in the same order for every role: for each block of rows,
// each pair of K tiles that some of its rows see; of those, the query tiles from
// the first that sees the pair's first token.
struct StWork {
    int j0, end;     // the range's first token, the end of its tokens that exist
    int kv, old;     // cached tokens; those that every query sees (causal)
    int rows, group, tiles, per, blocks, pairs;
    bool causal;
    __device__ __forceinline__ int first_row(int j) const {  // first row that sees token j (>= rows: none)
        const int64_t r = causal ? static_cast<int64_t>(max(0, j - old)) * group : 0;
        return static_cast<int>(min(r, static_cast<int64_t>(rows)));
    }
    __device__ __forceinline__ int first_tile(int rb, int pair) const {
        return max(rb * per, first_row(j0 + pair * 2 * kStTile) / kStTile);
    }
    __device__ __forceinline__ int end_tile(int rb) const { return min(tiles, rb * per + per); }
    __device__ __forceinline__ bool has(int rb, int pair) const {
        return first_row(j0 + pair * 2 * kStTile) < rows && first_tile(rb, pair) < end_tile(rb);
    }
    // the pair's second tile has tokens
    __device__ __forceinline__ bool second(int pair) const { return j0 + (2 * pair + 1) * kStTile < end; }
};

template <int D>
__global__ void __launch_bounds__(kStThreads, 1) paged_scores_tc_kernel(PagedScoreParams p, int range) {
    using Lay = StLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::kMisc);  // [0] tmem, [1] abort
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
    int b = blockIdx.x;
    const int h = b % p.g.kv_heads;
    b /= p.g.kv_heads;
    const int s = b % p.g.seqs;
    const int j0 = (b / p.g.seqs) * range;  // (range: a multiple of 256)
    if (j0 >= p.g.max_kv) return;
    const Seq q = load_seq(p.g, s);
    const int64_t row_at = (static_cast<int64_t>(s) * p.g.kv_heads + h) * p.score_stride;
    StWork w;
    w.j0 = j0;
    w.end = min(q.kv, j0 + range);
    w.kv = q.kv;
    w.old = q.kv - q.n;
    w.rows = q.n * p.group;
    w.group = p.group;
    w.causal = p.causal != 0;
    w.tiles = (w.rows + kStTile - 1) / kStTile;
    w.blocks = (w.tiles + kStQTiles - 1) / kStQTiles;
    w.per = w.blocks > 0 ? (w.tiles + w.blocks - 1) / w.blocks : 1;
    w.pairs = w.rows > 0 ? max(0, (w.end - j0 + 2 * kStTile - 1) / (2 * kStTile)) : 0;
    // tokens that no pair has keep their scores
    const int stop = min(p.g.max_kv, j0 + range);
    for (int j = j0 + w.pairs * 2 * kStTile + tid; j < stop; j += kStThreads) p.out[row_at + j] = p.scores[row_at + j];
    if (w.pairs == 0) return;
    AbortState ab{reinterpret_cast<volatile uint32_t*>(&misc[1]), p.g.status, p.wait_ns};

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars[S_K_FULL + i], 4);
            mbar_init(&bars[S_K_EMPTY + i], 1);
            mbar_init(&bars[S_S_FULL + i], 1);
            mbar_init(&bars[S_S_FREE + i], 4);
        }
        mbar_init(&bars[S_Q_FULL], 16);
        mbar_init(&bars[S_Q_EMPTY], 16);
        mbar_init(&bars[S_DRAIN], 2);
        misc[1] = 0u;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc[0], 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (wg == 0) {
        regs_dec<40>();
        if (warp < 2) {
            // -------------------------------------------------------- products
            const int g = warp;
            const uint32_t idesc = instr_desc(kFmtBF16, kFmtBF16, 128, 128);
            const uint64_t dk = smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2);
            const uint32_t hi = static_cast<uint32_t>(dk >> 32), k_lo = static_cast<uint32_t>(dk);
            const uint32_t q_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2));
            bool ok = true;
            // pairs of all groups; first, second K tiles and units of this one
            int pc = 0, ka_count = 0, kb_count = 0, uc[2] = {0, 0};
            for (int rb = 0; rb < w.blocks && ok; ++rb) {
                ok = warp_wait(&bars[S_Q_FULL], rb & 1, ab, kDevTimeoutMma);
                for (int pair = 0; pair < w.pairs && ok; ++pair) {
                    if (!w.has(rb, pair) || (pc++ & 1) != g) continue;
                    const int q0 = w.first_tile(rb, pair), q1 = w.end_tile(rb), tiles = w.second(pair) ? 2 : 1;
                    ok = warp_wait(&bars[S_K_FULL + 2 * g], ka_count++ & 1, ab, kDevTimeoutMma);
                    if (ok && tiles == 2) ok = warp_wait(&bars[S_K_FULL + 2 * g + 1], kb_count++ & 1, ab, kDevTimeoutMma);
                    for (int t = q0; t < q1 && ok; ++t) {
                        const uint32_t qb = q_lo + (t - rb * w.per) * (Lay::kTile >> 4);
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            if (a == tiles || !ok) break;
                            const int place = 2 * g + a;
                            ok = warp_wait(&bars[S_S_FREE + place], (uc[a]++ & 1) ^ 1, ab, kDevTimeoutMma);
                            tc_fence_after();
                            if (ok && elect_one()) {
                                const uint32_t d = tmem + 128u * place, ka = k_lo + place * (Lay::kTile >> 4);
                                mma_f16_ss_at<0, 0>(d, ka, qb, hi, idesc, 0);
                                mma_f16_ss_at<2, 2>(d, ka, qb, hi, idesc, 1);
                                mma_f16_ss_at<4, 4>(d, ka, qb, hi, idesc, 1);
                                mma_f16_ss_at<6, 6>(d, ka, qb, hi, idesc, 1);
                                if (D == 128) {
                                    mma_f16_ss_at<1024, 1024>(d, ka, qb, hi, idesc, 1);
                                    mma_f16_ss_at<1026, 1026>(d, ka, qb, hi, idesc, 1);
                                    mma_f16_ss_at<1028, 1028>(d, ka, qb, hi, idesc, 1);
                                    mma_f16_ss_at<1030, 1030>(d, ka, qb, hi, idesc, 1);
                                }
                                mma_commit(&bars[S_S_FULL + place]);
                                if (t + 1 == q1) mma_commit(&bars[S_K_EMPTY + place]);
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            // every product has finished before the tensor memory is released
            if (elect_one()) mma_commit(&bars[S_DRAIN]);
            __syncwarp();
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars[S_DRAIN], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else if (wg <= 4) {
        // ------------------------------------------------------------ sums
        regs_inc<80>();
        const int place = wg - 1, g = place >> 1, a = place & 1, quad = warp & 3;
        const int st = tid - 128;  // number among the groups' threads
        const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * place;
        const float2 c2 = make_float2(p.sm_log2, p.sm_log2);
        float* minus = reinterpret_cast<float*>(smem + Lay::kMinus);
        int pc = 0, n = 0;  // pairs, units of this group
        bool ok = true;
        for (int rb = 0; rb < w.blocks && ok; ++rb) {
            // the block's query rows: thread st has the piece st % kPieces of the
            // rows st / kPieces + i kRows; and lse of each row
            if (rb > 0) ok = warp_wait(&bars[S_Q_EMPTY], (rb - 1) & 1, ab, kDevTimeoutSoftmax);
            if (!ok) break;
            constexpr int kPieces = D / 8, kRows = kStSums / kPieces, kBatch = 6;
            const int first = rb * w.per * kStTile, count = (w.end_tile(rb) - rb * w.per) * kStTile;
            for (int r0 = st / kPieces; r0 < count; r0 += kBatch * kRows) {
                uint4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int rw = first + r0 + i * kRows;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (r0 + i * kRows < count && rw < w.rows) {
                        const int tok = p.group == 1 ? rw : rw / p.group, head = h * p.group + rw - tok * p.group;
                        v[i] = ldg_nc_na_v4(p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride +
                                            static_cast<int64_t>(head) * D + 8 * (st % kPieces));
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int row = r0 + i * kRows;
                    if (row < count)
                        *reinterpret_cast<uint4*>(smem + Lay::kQ + (row >> 7) * Lay::kTile +
                                                  bktile_off(row & 127, 8 * (st % kPieces))) =
                            make_uint4(__byte_perm(v[i].x, v[i].y, 0x5410), __byte_perm(v[i].x, v[i].y, 0x7632),
                                       __byte_perm(v[i].z, v[i].w, 0x5410), __byte_perm(v[i].z, v[i].w, 0x7632));
                }
            }
            for (int row = st; row < count; row += kStSums) {
                const int rw = first + row;
                float m = -INFINITY;  // rows past the last, and rows that saw nothing, add nothing
                if (rw < w.rows) {
                    const int tok = rw / p.group, head = h * p.group + rw - tok * p.group;
                    m = -__ldg(p.lse + static_cast<int64_t>(q.q0 + tok) * p.heads + head) * 1.4426950408889634f;
                    if (m == INFINITY) m = -INFINITY;
                }
                minus[row] = m;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_Q_FULL]);
            ok = warp_wait(&bars[S_Q_FULL], rb & 1, ab, kDevTimeoutSoftmax);
            for (int pair = 0; pair < w.pairs && ok; ++pair) {
                const int jp = j0 + pair * 2 * kStTile;
                const int j = jp + a * kStTile + quad * 32 + lane;  // the thread's token
                if (!w.has(rb, pair)) {
                    // no row of any block sees the pair
                    if (rb == 0 && g == 0 && w.first_row(jp) >= w.rows && j < stop) p.out[row_at + j] = p.scores[row_at + j];
                    continue;
                }
                if ((pc++ & 1) != g) continue;
                // the first block of rows that sees the pair starts from the given scores
                const float* from = rb == w.first_row(jp) / kStTile / w.per ? p.scores : p.out;
                float2 acc[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
                if (a == 0 || w.second(pair)) {
                    const int q0 = w.first_tile(rb, pair), q1 = w.end_tile(rb);
                    const int seen = w.first_row(j);  // the first row that sees the token
                    for (int t = q0; t < q1; ++t, ++n) {
                        ok = warp_wait(&bars[S_S_FULL + place], n & 1, ab, kDevTimeoutSoftmax);
                        if (!ok) break;
                        tc_fence_after();
                        const float* mt = minus + (t - rb * w.per) * kStTile;
                        const int lo = seen - t * kStTile;  // columns from this on count
                        const bool full = __all_sync(0xffffffffu, lo <= 0);
#pragma unroll 1
                        for (int c0 = 0; c0 < kStTile; c0 += 32) {
                            uint32_t v[32];
                            tmem_ld32(at + c0, v);
                            if (c0 + 32 == kStTile) {
                                // the scores are in registers: their place is free
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&bars[S_S_FREE + place]);
                            }
                            float2 x[16];
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                const float4 m = *reinterpret_cast<const float4*>(mt + c0 + 2 * k);
                                x[k] = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2,
                                            make_float2(m.x, m.y));
                                x[k + 1] = fma2(make_float2(__uint_as_float(v[2 * k + 2]), __uint_as_float(v[2 * k + 3])), c2,
                                                make_float2(m.z, m.w));
                            }
#pragma unroll
                            for (int k = 0; k < 16; ++k) x[k] = make_float2(ex2(x[k].x), ex2(x[k].y));
                            if (!full) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    if (c0 + 2 * k < lo) x[k].x = 0.f;
                                    if (c0 + 2 * k + 1 < lo) x[k].y = 0.f;
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 16; ++k) acc[k & 3] = add2(acc[k & 3], x[k]);
                        }
                    }
                    if (!ok) break;
                }
                if (j < stop) {
                    const float2 x = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                    p.out[row_at + j] = from[row_at + j] + (j < q.kv ? x.x + x.y : 0.f);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_Q_EMPTY]);
        }
    } else {
        // ------------------------------------------------------------ K
        // Each warpgroup has one tile of every pair.  Thread ct: the pieces of 16
        // dims ct % 4 (+ 4 in the second 64 dims) of the rows ct / 4 + 32 m.  Lane
        // l < 8 of a warp looks up the block of 16 tokens l of the tile.
        const int ct = tid & 127, a = wg - 5;
        constexpr int NB = D / 64;
        const int rr = ct >> 2, pb = p.g.page_shift - 4;
        const uint8_t* kbase = p.g.kcodes + (rr & 15) * D + 16 * (ct & 3);
        const uint8_t* sbase = p.g.kscale + (rr & 15);
        const uint32_t* table =
            reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
        uint4 kr[4 * NB];
        uint32_t ks[4];
        // the next pair with work after (rb, pair); pair = -1 starts; rb = blocks ends
        auto advance = [&](int& rb, int& pair) {
            do {
                if (++pair == w.pairs) {
                    pair = 0;
                    ++rb;
                }
            } while (rb < w.blocks && !w.has(rb, pair));
        };
        auto token = [&](int pair) { return j0 + (2 * pair + a) * kStTile + 16 * (lane & 7); };
        auto entry = [&](int rb, int pair) {
            const int t = token(pair);
            return rb < w.blocks && t < q.kv ? static_cast<int>(ldg_early(table + (t >> p.g.page_shift))) : 0;
        };
        // (blocks behind the end, or on a bad page, read block 0: their sums are not used)
        auto block_of = [&](int rb, int pair, int page) {
            const int t = token(pair);
            if (rb >= w.blocks || t >= q.kv) return 0u;
            const uint32_t at = static_cast<uint32_t>(check_page(p.g, page) ? page : 0) * p.g.kv_heads + h;
            return (at << pb) + (static_cast<uint32_t>(t >> 4) & ((1u << pb) - 1u));
        };
        auto fetch = [&](int m, uint32_t blk) {
            const uint64_t at = __shfl_sync(0xffffffffu, blk, (rr >> 4) + 2 * m);
#pragma unroll
            for (int x = 0; x < NB; ++x) kr[m * NB + x] = ldg_nc_na_v4(kbase + at * (16 * D) + 64 * x);
            ks[m] = ldg_early(sbase + at * 16);
        };
        int rb = 0, pair = -1, pc = 0;
        int uses[2] = {0, 0};  // of each buffer of the tile so far
        advance(rb, pair);
        int rb1 = rb, pair1 = pair;
        if (rb < w.blocks) {
            const uint32_t blk = block_of(rb, pair, entry(rb, pair));
#pragma unroll
            for (int m = 0; m < 4; ++m) fetch(m, blk);
            advance(rb1, pair1);
        }
        int ahead = entry(rb1, pair1);
        bool ok = true;
        while (ok && rb < w.blocks) {
            const uint32_t blk = block_of(rb1, pair1, ahead);
            int rb2 = rb1, pair2 = pair1;
            if (rb1 < w.blocks) advance(rb2, pair2);
            ahead = entry(rb2, pair2);
            const bool there = a == 0 || w.second(pair);
            const int buf = 2 * (pc & 1) + a;  // (the group of the pair, the tile of the pair)
            if (there) ok = warp_wait(&bars[S_K_EMPTY + buf], (uses[pc & 1]++ & 1) ^ 1, ab, kDevTimeoutConvert);
            uint8_t* dst = smem + Lay::kK + buf * Lay::kTile;
            uint8_t* lo = dst + bktile_off(rr, 16 * (ct & 3));
            uint8_t* hi = dst + bktile_off(rr, 16 * (ct & 3) + 8);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (ok && there) {
                    const uint32_t f1 = scale_factor(ks[m]);
                    const uint32_t f[8] = {f1, f1, f1, f1, f1, f1, f1, f1};
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        const int off = x * (kStTile * 128) + m * (32 * 128);
                        put16(lo + off, hi + off, kr[m * NB + x], f);
                    }
                }
                fetch(m, blk);  // the next pair's rows, into the registers just freed
            }
            if (ok && there) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[S_K_FULL + buf]);
            }
            ++pc;
            rb = rb1;
            pair = pair1;
            rb1 = rb2;
            pair1 = pair2;
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch_d(const PagedScoreParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    constexpr uint32_t smem = StLayout<D>::kAlloc;
    static_assert(smem <= 227 * 1024, "shared memory over the sm_103 limit");
    cudaError_t e = smem_limit_once(paged_scores_tc_kernel<D>, smem, configured);
    if (e != cudaSuccess) return e;
    // Ranges of cached tokens: as many blocks as fill the SMs once (a block's
    // set-up takes as long as several tiles: one sequence of 8,000 tokens x 8 KV
    // heads, 128 ranges of two tiles 15.6 us, 256 of one 22.7), at least two
    // tiles each.
    const int64_t rows = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    const int64_t pairs = (p.g.max_kv + 255) / 256;
    const int64_t ranges = std::min<int64_t>(pairs, std::max<int64_t>(1, 152 / rows));
    const int range = static_cast<int>((pairs + ranges - 1) / ranges) * 256;
    const int64_t blocks = (p.g.max_kv + range - 1) / range * rows;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    paged_scores_tc_kernel<D><<<static_cast<unsigned>(blocks), kStThreads, smem, s>>>(p, range);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_scores_tc(const PagedScoreParams& p, int D, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
