// rc_paged_scores_tc.cu -- the attention weight of each cached token, for many
// query rows, on the tensor cores (tcgen05).
//
// Transposed: S^T = K Q^T, so a thread holds one cached token's scores (a lane of
// TMEM) and its sum over the queries runs in one register, in one order; no two
// threads add to one entry.  A block has a range of the cached tokens of one
// (sequence, KV head) and goes over the head's query rows in blocks of up to
// 384, which stay in shared memory as three tiles while the cached tokens stream
// past, two tiles of 128 at a time (one for each group of four warps):
//   warp 0         issues the products (one lane) and owns TMEM: four places of
//                  128 x 128 scores, two a group, so that the products of a
//                  group's next tile run while it sums this one
//   warps 4 .. 11  groups 0 and 1: exp2(S c - lse) and the sum over the columns
//   warps 12 .. 19 read K's codes from the pages (a pair of tiles ahead, in
//                  registers), make them bf16 operand tiles (two pairs of
//                  buffers), and bring the query rows
// With the queries kept, K is read and converted once per 384 rows, and the
// queries once per block: keeping K instead would read them for every 128
// tokens (430 MB of cache traffic for 757 x 5,788 tokens x 48 heads).
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kStThreads = 640;
constexpr int kStTile = 128;
constexpr int kStQTiles = 3;  // query tiles in shared memory
constexpr int kStConvert = 256;

enum : int {
    S_K_FULL = 0,    // [4] buffer 2 (tile of the group & 1) + group: K tile converted
    S_K_EMPTY = 4,   // [4] its products have finished
    S_S_FULL = 8,    // [4] place 2 group + (unit & 1): scores in TMEM
    S_S_FREE = 12,   // [4] the group has read them
    S_Q_FULL = 16,   // the block's query rows are in place
    S_Q_EMPTY = 17,  // products and groups are done with them
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
            mbar_init(&bars[S_K_FULL + i], 8);
            mbar_init(&bars[S_K_EMPTY + i], 1);
            mbar_init(&bars[S_S_FULL + i], 1);
            mbar_init(&bars[S_S_FREE + i], 4);
        }
        mbar_init(&bars[S_Q_FULL], 8);
        mbar_init(&bars[S_Q_EMPTY], 1 + 8);
        mbar_init(&bars[S_DRAIN], 1);
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

    if (warp == 0) {
        // ------------------------------------------------------------ products
        const uint32_t idesc = instr_desc(kFmtBF16, kFmtBF16, 128, 128);
        const uint64_t dk = smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2);
        const uint32_t hi = static_cast<uint32_t>(dk >> 32), k_lo = static_cast<uint32_t>(dk);
        const uint32_t q_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2));
        bool ok = true;
        int kc[2] = {0, 0}, uc[2] = {0, 0};  // K tiles, units of each group so far
        for (int rb = 0; rb < w.blocks && ok; ++rb) {
            ok = warp_wait(&bars[S_Q_FULL], rb & 1, ab, kDevTimeoutMma);
            for (int pair = 0; pair < w.pairs && ok; ++pair) {
                if (!w.has(rb, pair)) continue;
                const int q0 = w.first_tile(rb, pair), q1 = w.end_tile(rb), groups = w.second(pair) ? 2 : 1;
                for (int g = 0; g < groups && ok; ++g)
                    ok = warp_wait(&bars[S_K_FULL + 2 * (kc[g] & 1) + g], (kc[g] >> 1) & 1, ab, kDevTimeoutMma);
                for (int t = q0; t < q1 && ok; ++t)
                    for (int g = 0; g < groups && ok; ++g) {
                        const int n = g == 0 ? uc[0]++ : uc[1]++, place = 2 * g + (n & 1);
                        ok = warp_wait(&bars[S_S_FREE + place], ((n >> 1) & 1) ^ 1, ab, kDevTimeoutMma);
                        tc_fence_after();
                        const int buf = 2 * (kc[g] & 1) + g;
                        if (ok && elect_one()) {
                            const uint32_t d = tmem + 128u * place;
                            const uint32_t ka = k_lo + buf * (Lay::kTile >> 4);
                            const uint32_t qb = q_lo + (t - rb * w.per) * (Lay::kTile >> 4);
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
                            if (t + 1 == q1) mma_commit(&bars[S_K_EMPTY + buf]);
                        }
                        __syncwarp();
                    }
                ++kc[0];
                kc[1] += groups - 1;
            }
            if (elect_one()) mma_commit(&bars[S_Q_EMPTY]);
            __syncwarp();
        }
        // every product has finished before the tensor memory is released
        if (elect_one()) mma_commit(&bars[S_DRAIN]);
        __syncwarp();
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&bars[S_DRAIN], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
    } else if (wg == 1 || wg == 2) {
        // ------------------------------------------------------------ sums
        const int g = wg - 1, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t at0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 256u * g;
        const float c = p.sm_log2;
        const float2 c2 = make_float2(c, c);
        const float* minus = reinterpret_cast<const float*>(smem + Lay::kMinus);
        int n = 0;  // units so far
        bool ok = true;
        for (int rb = 0; rb < w.blocks && ok; ++rb) {
            // (lse of the rows: written with the query tiles)
            ok = warp_wait(&bars[S_Q_FULL], rb & 1, ab, kDevTimeoutSoftmax);
            for (int pair = 0; pair < w.pairs && ok; ++pair) {
                const int j = j0 + (2 * pair + g) * kStTile + r;  // the thread's token
                const bool mine = j < stop;
                if (!w.has(rb, pair) || (g == 1 && !w.second(pair))) {
                    // no row of any block sees the pair, or its second tile is empty
                    if (rb == 0 && (w.first_row(j0 + pair * 2 * kStTile) >= w.rows || (g == 1 && !w.second(pair))) && mine)
                        p.out[row_at + j] = p.scores[row_at + j];
                    continue;
                }
                const int q0 = w.first_tile(rb, pair), q1 = w.end_tile(rb);
                const int first = w.first_row(j);  // the first row that sees the token
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                for (int t = q0; t < q1 && ok; ++t, ++n) {
                    ok = warp_wait(&bars[S_S_FULL + 2 * g + (n & 1)], (n >> 1) & 1, ab, kDevTimeoutSoftmax);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = at0 + 128u * (n & 1);
                    const float* mt = minus + (t - rb * w.per) * kStTile;
                    // columns of the tile that count: rows [first, rows)
                    const int lo = first - t * kStTile, hi = w.rows - t * kStTile;
                    const bool full = __all_sync(0xffffffffu, lo <= 0 && hi >= kStTile);
                    uint32_t va[32], vb[32];
                    auto add = [&](uint32_t (&v)[32], int c0) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(mt + c0 + k);
                            const float2 x0 = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2,
                                                   make_float2(m.x, m.y));
                            const float2 x1 = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), c2,
                                                   make_float2(m.z, m.w));
                            v[k] = __float_as_uint(ex2(x0.x));
                            v[k + 1] = __float_as_uint(ex2(x0.y));
                            v[k + 2] = __float_as_uint(ex2(x1.x));
                            v[k + 3] = __float_as_uint(ex2(x1.y));
                        }
                        if (!full) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (c0 + k < lo || c0 + k >= hi) v[k] = 0u;
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            acc[(k >> 1) & 3] =
                                add2(acc[(k >> 1) & 3], make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                    };
                    tmem_ld32_async(at, va);
#pragma unroll 1
                    for (int c0 = 0; c0 < kStTile; c0 += 64) {
                        tmem_wait_ld_dep(va);
                        tmem_ld32_async(at + c0 + 32, vb);
                        add(va, c0);
                        tmem_wait_ld_dep(vb);
                        if (c0 + 64 < kStTile) tmem_ld32_async(at + c0 + 64, va);
                        if (c0 + 64 == kStTile) {
                            // the scores are in registers: their place is free
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bars[S_S_FREE + 2 * g + (n & 1)]);
                        }
                        add(vb, c0 + 32);
                    }
                }
                if (!ok) break;
                if (mine) {
                    const float2 a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                    // the first block of rows that sees the pair starts from the given scores
                    const bool begin = rb == (w.first_row(j0 + pair * 2 * kStTile) / kStTile) / w.per;
                    const float old = begin ? p.scores[row_at + j] : p.out[row_at + j];
                    p.out[row_at + j] = old + (j < q.kv ? a.x + a.y : 0.f);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_Q_EMPTY]);
        }
    } else if (wg >= 3) {
        // ------------------------------------------------------------ K and Q
        // Thread ct: the pieces of 16 dims ct % 4 (+ 4 in the second 64 dims) of
        // the rows ct / 4 and ct / 4 + 64 of each tile.  Lane l < 16 of a warp
        // looks up the block of 16 tokens l of the pair.
        const int ct = tid - 3 * 128;
        constexpr int NB = D / 64;
        const int rr = ct >> 2, pb = p.g.page_shift - 4;
        const uint8_t* kbase = p.g.kcodes + (rr & 15) * D + 16 * (ct & 3);
        const uint8_t* sbase = p.g.kscale + (rr & 15);
        const uint32_t* table =
            reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
        uint4 kr[2][2 * NB];
        uint32_t ks[2][2];
        // the next pair with work after (rb, pair); pair = -1 starts; rb = blocks ends
        auto advance = [&](int& rb, int& pair) {
            do {
                if (++pair == w.pairs) {
                    pair = 0;
                    ++rb;
                }
            } while (rb < w.blocks && !w.has(rb, pair));
        };
        auto entry = [&](int rb, int pair) {
            const int t = j0 + pair * 2 * kStTile + 16 * (lane & 15);
            return rb < w.blocks && t < q.kv ? static_cast<int>(ldg_early(table + (t >> p.g.page_shift))) : 0;
        };
        // (blocks behind the end, or on a bad page, read block 0: their sums are not used)
        auto block_of = [&](int rb, int pair, int page) {
            const int t = j0 + pair * 2 * kStTile + 16 * (lane & 15);
            if (rb >= w.blocks || t >= q.kv) return 0u;
            const uint32_t at = static_cast<uint32_t>(check_page(p.g, page) ? page : 0) * p.g.kv_heads + h;
            return (at << pb) + (static_cast<uint32_t>(t >> 4) & ((1u << pb) - 1u));
        };
        auto fetch = [&](int g, uint32_t blk) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint64_t at = __shfl_sync(0xffffffffu, blk, 8 * g + (rr >> 4) + 4 * m);
#pragma unroll
                for (int x = 0; x < NB; ++x) kr[g][m * NB + x] = ldg_nc_na_v4(kbase + at * (16 * D) + 64 * x);
                ks[g][m] = ldg_early(sbase + at * 16);
            }
        };
        int rb = 0, pair = -1, kc[2] = {0, 0};
        advance(rb, pair);
        int rb1 = rb, pair1 = pair;
        if (rb < w.blocks) {
            const uint32_t blk = block_of(rb, pair, entry(rb, pair));
            fetch(0, blk);
            fetch(1, blk);
            advance(rb1, pair1);
        }
        int ahead = entry(rb1, pair1);
        bool ok = true;
        int loaded = -1;  // the block of rows in shared memory
        while (ok) {
            // query rows up to the current pair's block (blocks without work are passed as well)
            for (const int want = min(rb, w.blocks - 1); loaded < want && ok;) {
                ++loaded;
                if (loaded > 0) ok = warp_wait(&bars[S_Q_EMPTY], (loaded - 1) & 1, ab, kDevTimeoutConvert);
                if (!ok) break;
                constexpr int kPieces = D / 8;
                const int first = loaded * w.per * kStTile, count = (w.end_tile(loaded) - loaded * w.per) * kStTile;
                for (int u = ct; u < count * kPieces; u += kStConvert) {
                    const int row = u / kPieces, c = u % kPieces, rw = first + row;
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (rw < w.rows) {
                        const int tok = rw / p.group, head = h * p.group + rw - tok * p.group;
                        v = ldg_nc_na_v4(p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D +
                                         8 * c);
                    }
                    *reinterpret_cast<uint4*>(smem + Lay::kQ + (row >> 7) * Lay::kTile + bktile_off(row & 127, 8 * c)) =
                        make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                                   __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
                }
                for (int row = ct; row < count; row += kStConvert) {
                    const int rw = first + row;
                    float m = 0.f;
                    if (rw < w.rows) {
                        const int tok = rw / p.group, head = h * p.group + rw - tok * p.group;
                        m = -__ldg(p.lse + static_cast<int64_t>(q.q0 + tok) * p.heads + head) * 1.4426950408889634f;
                        if (m == INFINITY) m = -INFINITY;  // a row that saw nothing adds nothing
                    }
                    reinterpret_cast<float*>(smem + Lay::kMinus)[row] = m;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[S_Q_FULL]);
            }
            if (!ok || rb >= w.blocks) break;
            const uint32_t blk = block_of(rb1, pair1, ahead);
            int rb2 = rb1, pair2 = pair1;
            if (rb1 < w.blocks) advance(rb2, pair2);
            ahead = entry(rb2, pair2);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (ok && (g == 0 || w.second(pair))) {
                    const int buf = 2 * (kc[g] & 1) + g;
                    ok = warp_wait(&bars[S_K_EMPTY + buf], ((kc[g] >> 1) & 1) ^ 1, ab, kDevTimeoutConvert);
                    ++kc[g];
                    if (ok) {
                        uint8_t* dst = smem + Lay::kK + buf * Lay::kTile;
                        uint8_t* lo = dst + bktile_off(rr, 16 * (ct & 3));
                        uint8_t* hi = dst + bktile_off(rr, 16 * (ct & 3) + 8);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint32_t f1 = scale_factor(ks[g][m]);
                            const uint32_t f[8] = {f1, f1, f1, f1, f1, f1, f1, f1};
#pragma unroll
                            for (int x = 0; x < NB; ++x) {
                                const int off = x * (kStTile * 128) + m * (64 * 128);
                                put16(lo + off, hi + off, kr[g][m * NB + x], f);
                            }
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[S_K_FULL + buf]);
                    }
                }
                fetch(g, blk);
            }
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
    // set-up takes as long as several tiles), at least two tiles each.
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
