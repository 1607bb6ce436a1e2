// rc_paged_scores_tc.cu -- the attention weight of each cached token, for many
// query rows, on the tensor cores (tcgen05).
//
// Transposed: S^T = K Q^T, so a thread holds one cached token's scores (a lane of
// TMEM).  A block has a range of the cached tokens of one (sequence, KV head) and
// goes over the head's query rows in blocks of up to 768, which stay in shared
// memory as six tiles while the cached tokens stream past in tiles of 128.  The
// operand with the cached tokens is in TMEM, not in shared memory: each thread of
// the converters has a token's row, which is a lane there.
//   warp 0         issues the products (one lane) and owns TMEM: three places of
//                  128 x 128 scores and two K tiles
//   warps 4 .. 15  three groups, one a place: exp2(S c - lse) and the sum over the
//                  columns, a token a thread.  The units (K tile, query tile) go
//                  to the groups in turn; a group's sums of a pair of K tiles are put in
//                  shared memory, and the groups take turns in adding the three
//                  up, always in the same order: no two threads add to one entry.
//                  They also bring the query rows (by cp.async), and zeros in the place of
//                  those whose lse is -infinity: whatever they hold adds nothing.
//   warps 16 .. 23 read K's codes from the pages (a warpgroup's next tile is in its
//                  registers), make them bf16 (exactly: scales are powers of two)
//                  and put them in TMEM, a tile a warpgroup
// With the queries kept, K is read and converted once per 768 rows, and the
// queries once per block: keeping K instead would read them for every 128
// tokens (430 MB of cache traffic for 757 x 5,788 tokens x 48 heads).
//
// 757 queries x 5,788 tokens x 48 heads x 128: 57.2 us, 0.94 PFLOP/s, half of
// what a library product of bf16 matrices reaches.  Of the 126,000 cycles of a
// block 12,000 bring the queries; then a unit takes 1,000 where its product needs
// 530 and its exponentials 510: bound by the chain of a group (wait for the
// product, 64 columns to registers, exponentials, the other 64, the place handed
// back), of which shared memory and TMEM have room for three.  With K in shared
// memory, 384 rows at a time and four groups it took 71 us.
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

// 768 threads launched with 80 registers each; the warpgroups share them
// 32 + 3 x 112 + 2 x 56 = 6 x 80.
constexpr int kStThreads = 768;
constexpr int kStGroups = 3;
constexpr int kStSums = 128 * kStGroups;  // threads of the groups
constexpr int kStTile = 128;
constexpr int kStQTiles = 6;  // query tiles in shared memory
constexpr int kStParts = 4;   // pairs of K tiles whose sums are in shared memory
constexpr int kStPair = 2 * kStTile;
constexpr uint32_t kStTmemK = 128 * kStGroups;

enum : int {
    S_K_FULL = 0,      // [2] K tile converted
    S_K_EMPTY = 2,     // [2] its products have finished
    S_S_FULL = 4,      // [3] scores of a unit in TMEM
    S_S_FREE = 7,      // [3] the group has read them
    S_PART_FULL = 10,  // [4] every group's sums of a pair of K tiles are in place
    S_PART_EMPTY = 14, // [4] they have been added up
    S_Q_FULL = 18,     // the block's query rows and their lse are in place
    S_Q_EMPTY = 19,    // every group and the product warp are through with them
    S_Q_READY = 20,    // queries of rows that add nothing are zeros
    S_DRAIN = 21,
    S_COUNT = 22
};

template <int D>
struct StLayout {
    static constexpr uint32_t kTile = kStTile * D * 2;
    static constexpr uint32_t kQ = 0;                           // [6]
    static constexpr uint32_t kMinus = kQ + kStQTiles * kTile;  // fp32 [6][128]: -lse log2(e)
    static constexpr uint32_t kPart = kMinus + kStQTiles * kStTile * 4;  // fp32 [4][3][256]
    static constexpr uint32_t kBar = kPart + kStParts * kStGroups * kStPair * 4;
    static constexpr uint32_t kMisc = kBar + 8 * S_COUNT;
    static constexpr uint32_t kTotal = kMisc + 16;
    static constexpr uint32_t kAlloc = kTotal + 1024;
};

// What a block does, in the same order for every role: for each block of rows,
// each K tile that some of its rows see; of those, the query tiles from the first
// that sees the K tile's first token.
template <bool CAUSAL>
struct StWork {
    int j0, end;  // the range's first token, the end of its tokens that exist
    int old, n;   // tokens that every query sees (causal), new tokens
    int rows, group, tiles, per, blocks, ktiles;
    __device__ __forceinline__ int first_row(int j) const {  // first row that sees token j (>= rows: none)
        if (!CAUSAL || j <= old) return 0;
        return j - old < n ? (j - old) * group : rows;
    }
    __device__ __forceinline__ int first_tile(int rb, int i) const {
        if (!CAUSAL) return rb * per;
        return max(rb * per, first_row(j0 + i * kStTile) / kStTile);
    }
    __device__ __forceinline__ int end_tile(int rb) const { return min(tiles, rb * per + per); }
    __device__ __forceinline__ bool has(int rb, int i) const {
        return !CAUSAL || (first_row(j0 + i * kStTile) < rows && first_tile(rb, i) < end_tile(rb));
    }
};

// A cached token that is not a number also meets rows that add nothing and those
// past the last: its sum counts only if some other row of the block of rows sees
// it.  (Out of line: what a rare call needs is not kept in registers otherwise.)
template <bool CAUSAL>
__device__ __noinline__ float checked_sum(float sum, const float* minus, const StWork<CAUSAL>& w, int rb, int token) {
    if (sum == sum) return sum;
    const int first = rb * w.per * kStTile, end = min(w.end_tile(rb) * kStTile, w.rows);
    for (int row = max(first, w.first_row(token)); row < end; ++row)
        if (minus[row - first] != -INFINITY) return sum;
    return 0.f;
}

// Zeros in the place of the queries of rows st and st + kStSums, if they add nothing.
template <int D>
__device__ __noinline__ void zero_queries(uint8_t* smem, const float* minus, int st, int rows) {
    for (int row = st; row < rows; row += kStSums)
        if (minus[row] == -INFINITY)
            for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<uint4*>(smem + StLayout<D>::kQ + (row >> 7) * StLayout<D>::kTile + bktile_off(row & 127, 8 * k)) =
                    make_uint4(0, 0, 0, 0);
}

template <int D, bool CAUSAL>
__global__ void __launch_bounds__(kStThreads, 1) paged_scores_tc_kernel(PagedScoreParams p, int range) {
    using Lay = StLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::kMisc);  // [0] tmem, [1] abort, [2], [3] zeros are to be put
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2, quad = warp & 3;
    int b = blockIdx.x;
    const int h = b % p.g.kv_heads;
    b /= p.g.kv_heads;
    const int s = b % p.g.seqs;
    const int j0 = (b / p.g.seqs) * range;  // (range: a multiple of 128)
    if (j0 >= p.g.max_kv) return;
    const Seq q = load_seq(p.g, s);
    const int64_t row_at = (static_cast<int64_t>(s) * p.g.kv_heads + h) * p.score_stride;
    StWork<CAUSAL> w;
    w.j0 = j0;
    w.end = min(q.kv, j0 + range);
    w.old = q.kv - q.n;
    w.n = q.n;
    w.rows = q.n * p.group;
    w.group = p.group;
    w.tiles = (w.rows + kStTile - 1) / kStTile;
    w.blocks = (w.tiles + kStQTiles - 1) / kStQTiles;
    w.per = w.blocks > 0 ? (w.tiles + w.blocks - 1) / w.blocks : 1;
    w.ktiles = w.rows > 0 ? max(0, (w.end - j0 + kStTile - 1) / kStTile) : 0;
    // tokens behind the end keep their scores
    const int stop = min(p.g.max_kv, j0 + range);
    for (int j = (w.ktiles > 0 ? w.end : j0) + tid; j < stop; j += kStThreads) p.out[row_at + j] = p.scores[row_at + j];
    if (w.ktiles == 0) return;
    AbortState ab{reinterpret_cast<volatile uint32_t*>(&misc[1]), p.g.status, p.wait_ns};

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[S_K_FULL + i], 4);
            mbar_init(&bars[S_K_EMPTY + i], 1);
        }
        for (int i = 0; i < kStGroups; ++i) {
            mbar_init(&bars[S_S_FULL + i], 1);
            mbar_init(&bars[S_S_FREE + i], 4);
        }
        for (int i = 0; i < kStParts; ++i) {
            mbar_init(&bars[S_PART_FULL + i], kStSums / 32);
            mbar_init(&bars[S_PART_EMPTY + i], 4);
        }
        mbar_init(&bars[S_Q_FULL], kStSums / 32);
        mbar_init(&bars[S_Q_READY], kStSums / 32);
        mbar_init(&bars[S_Q_EMPTY], kStSums / 32 + 1);
        mbar_init(&bars[S_DRAIN], 1);
        misc[1] = misc[2] = misc[3] = 0u;
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
        regs_dec<32>();
        if (warp == 0) {
            // -------------------------------------------------------- products
            const uint32_t idesc = instr_desc(kFmtBF16, kFmtBF16, 128, 128);
            const uint64_t dq = smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2);
            const uint32_t hi = static_cast<uint32_t>(dq >> 32), q_lo = static_cast<uint32_t>(dq);
            bool ok = true;
            int kc = 0, place = 0, phase = 0;  // K tiles; the unit's place and how often it was used before
            for (int rb = 0; rb < w.blocks && ok; ++rb) {
                ok = warp_wait(&bars[S_Q_READY], rb & 1, ab, kDevTimeoutMma);
                for (int i = 0; i < w.ktiles && ok; ++i) {
                    if (!w.has(rb, i)) continue;
                    const int q0 = w.first_tile(rb, i), q1 = w.end_tile(rb), buf = kc & 1;
                    ok = warp_wait(&bars[S_K_FULL + buf], (kc >> 1) & 1, ab, kDevTimeoutMma);
                    for (int t = q0; t < q1 && ok; ++t) {
                        ok = warp_wait(&bars[S_S_FREE + place], (phase & 1) ^ 1, ab, kDevTimeoutMma);
                        tc_fence_after();
                        if (ok && elect_one()) {
                            const uint32_t d = tmem + 128u * place, ka = tmem + kStTmemK + (D / 2) * buf;
                            const uint32_t qb = q_lo + (t - rb * w.per) * (Lay::kTile >> 4);
                            mma_f16_ts_at<0, 0>(d, ka, qb, hi, idesc, 0);
                            mma_f16_ts_at<8, 2>(d, ka, qb, hi, idesc, 1);
                            mma_f16_ts_at<16, 4>(d, ka, qb, hi, idesc, 1);
                            mma_f16_ts_at<24, 6>(d, ka, qb, hi, idesc, 1);
                            if (D == 128) {
                                mma_f16_ts_at<32, 1024>(d, ka, qb, hi, idesc, 1);
                                mma_f16_ts_at<40, 1026>(d, ka, qb, hi, idesc, 1);
                                mma_f16_ts_at<48, 1028>(d, ka, qb, hi, idesc, 1);
                                mma_f16_ts_at<56, 1030>(d, ka, qb, hi, idesc, 1);
                            }
                            mma_commit(&bars[S_S_FULL + place]);
                            if (t + 1 == q1) mma_commit(&bars[S_K_EMPTY + buf]);
                        }
                        __syncwarp();
                        if (++place == kStGroups) {
                            place = 0;
                            ++phase;
                        }
                    }
                    ++kc;
                }
                // (a block of rows that sees none of the range has no products: without this the
                // groups could be two blocks ahead, and the wait above take one phase for another)
                if (ok && lane == 0) mbar_arrive(&bars[S_Q_EMPTY]);
            }
            // every product has finished before the tensor memory is released
            if (elect_one()) mma_commit(&bars[S_DRAIN]);
            __syncwarp();
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars[S_DRAIN], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else if (wg <= kStGroups) {
        // ------------------------------------------------------------ sums
        regs_inc<112>();
        const int g = wg - 1;
        const int st = tid - 128;  // number among the groups' threads
        const uint32_t at = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * g;
        const float2 c2 = make_float2(p.sm_log2, p.sm_log2);
        float* minus = reinterpret_cast<float*>(smem + Lay::kMinus);
        float* part = reinterpret_cast<float*>(smem + Lay::kPart) + quad * 32 + lane;
        // pairs of K tiles; units of this group; whose turn the next unit is (0:
        // this group's); whose the next pair is
        int pc = 0, n = 0, turn = g, mine = g;
        int last = 0;                // the pair that this group has still to add up: its first token here
        bool due = false;
        float old[2] = {0.f, 0.f};  // and its scores so far
        bool ok = true;
        // adds up the sums of the pair number k
        auto join = [&](int k, int rb) {
            const int slot = k & (kStParts - 1);
            ok = warp_wait(&bars[S_PART_FULL + slot], (k / kStParts) & 1, ab, kDevTimeoutEpilogue);
            if (!ok) return;
            const float* x = part + slot * (kStGroups * kStPair);
            float sum[2];
#pragma unroll
            for (int a = 0; a < 2; ++a, x += kStTile) sum[a] = (x[0] + x[kStPair]) + x[2 * kStPair];
            // a cached token that is not a number also meets rows that add nothing, and those
            // past the last
            if (__any_sync(0xffffffffu, sum[0] + sum[1] != sum[0] + sum[1])) {
#pragma unroll
                for (int a = 0; a < 2; ++a) sum[a] = checked_sum<CAUSAL>(sum[a], minus, w, rb, last + a * kStTile);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_PART_EMPTY + slot]);
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const int j = last + a * kStTile;
                if (j < w.end) p.out[row_at + j] = old[a] + sum[a];
            }
            due = false;
        };
        for (int rb = 0; rb < w.blocks && ok; ++rb) {
            // the block's query rows: thread st has the piece st % kPieces of the
            // rows st / kPieces + i kRows; and lse of each row
            if (rb > 0) ok = warp_wait(&bars[S_Q_EMPTY], (rb - 1) & 1, ab, kDevTimeoutSoftmax);
            if (!ok) break;
            constexpr int kPieces = D / 8, kRows = kStSums / kPieces;
            const int first = rb * w.per * kStTile, count = (w.end_tile(rb) - rb * w.per) * kStTile;
#pragma unroll 4
            for (int row = st / kPieces; row < count; row += kRows) {
                const int rw = first + row, tok = p.group == 1 ? rw : rw / p.group, head = h * p.group + rw - tok * p.group;
                const bool have = rw < w.rows;
                const __nv_bfloat16* src =
                    have ? p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D : p.q;
                cp_async16_or_zero(smem + Lay::kQ + (row >> 7) * Lay::kTile + bktile_off(row & 127, 8 * (st % kPieces)),
                                   src + 8 * (st % kPieces), have);
            }
            // Queries of rows that add nothing (lse -infinity) become zeros, as what they hold
            // may not be numbers.  Whether there are such rows is known once every warp's are
            // in place (word rb & 1; the other is free until the next block of rows).
            volatile uint32_t* marks = misc + 2;
            for (int row = st; row < count; row += kStSums) {
                const int rw = first + row;
                float m = -INFINITY;  // rows past the last, and rows that saw nothing, add nothing
                if (rw < w.rows) {
                    const int tok = rw / p.group, head = h * p.group + rw - tok * p.group;
                    m = -__ldg(p.lse + static_cast<int64_t>(q.q0 + tok) * p.heads + head) * 1.4426950408889634f;
                    if (m == INFINITY) {
                        m = -INFINITY;
                        marks[rb & 1] = 1u;
                    }
                }
                minus[row] = m;
            }
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_Q_FULL]);
            ok = warp_wait(&bars[S_Q_FULL], rb & 1, ab, kDevTimeoutSoftmax);
            if (ok && marks[rb & 1] != 0u) {
                zero_queries<D>(smem, minus, st, min(count, w.rows - first));
                fence_async_smem();
            }
            if (st == 0) marks[(rb & 1) ^ 1] = 0u;
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&bars[S_Q_READY]);
            for (int i = 0; i < w.ktiles && ok; i += 2) {
                const int jt = j0 + i * kStTile, j = jt + quad * 32 + lane;  // the pair's first token, the thread's first
                if (!w.has(rb, i)) continue;
                float next_old[2] = {0.f, 0.f};
                if (mine == 0) {
                    // the first block of rows that sees the tile starts from the given scores
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float* from = rb == 0 || w.first_row(jt + a * kStTile) >= rb * w.per * kStTile ? p.scores : p.out;
                        if (j + a * kStTile < w.end) next_old[a] = from[row_at + j + a * kStTile];
                    }
                }
                const int slot = pc & (kStParts - 1);
                ok = warp_wait(&bars[S_PART_EMPTY + slot], ((pc / kStParts) & 1) ^ 1, ab, kDevTimeoutEpilogue);
                // this group's share of the pair, a tile at a time
#pragma unroll 1
                for (int a = 0; a < 2 && ok; ++a) {
                    float2 acc[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.f, 0.f);
                    const bool there = i + a < w.ktiles && (a == 0 || w.has(rb, i + a));
                    const int q0 = there ? w.first_tile(rb, i + a) : 0, q1 = there ? w.end_tile(rb) : 0;
                    const int seen = w.first_row(j + a * kStTile);  // the first row that sees the token
                    for (int t = q0; t < q1; ++t) {
                        const bool ours = turn == 0;
                        turn = turn == 0 ? kStGroups - 1 : turn - 1;
                        if (!ours) continue;
                        ok = warp_wait(&bars[S_S_FULL + g], n++ & 1, ab, kDevTimeoutSoftmax);
                        if (!ok) break;
                        tc_fence_after();
                        const float* mt = minus + (t - rb * w.per) * kStTile;
                        const int lo = seen - t * kStTile;  // columns from this on count
                        const bool full = !CAUSAL || __all_sync(0xffffffffu, lo <= 0);
#pragma unroll 1
                        for (int c0 = 0; c0 < kStTile; c0 += 64) {
                            uint32_t v[64];
                            tmem_ld64(at + c0, v);
                            if (c0 != 0) {
                                // the scores are in registers: their place is free
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&bars[S_S_FREE + g]);
                            }
#pragma unroll
                            for (int c = 0; c < 64; c += 16) {
                                float2 x[8];
#pragma unroll
                                for (int k = 0; k < 8; k += 2) {
                                    const float4 m = *reinterpret_cast<const float4*>(mt + c0 + c + 2 * k);
                                    x[k] = fma2(make_float2(__uint_as_float(v[c + 2 * k]), __uint_as_float(v[c + 2 * k + 1])), c2,
                                                make_float2(m.x, m.y));
                                    x[k + 1] = fma2(make_float2(__uint_as_float(v[c + 2 * k + 2]), __uint_as_float(v[c + 2 * k + 3])),
                                                    c2, make_float2(m.z, m.w));
                                }
#pragma unroll
                                for (int k = 0; k < 8; ++k) x[k] = make_float2(ex2(x[k].x), ex2(x[k].y));
                                if (!full) {
#pragma unroll
                                    for (int k = 0; k < 8; ++k) {
                                        if (c0 + c + 2 * k < lo) x[k].x = 0.f;
                                        if (c0 + c + 2 * k + 1 < lo) x[k].y = 0.f;
                                    }
                                }
#pragma unroll
                                for (int k = 0; k < 8; ++k) acc[k & 3] = add2(acc[k & 3], x[k]);
                            }
                        }
                    }
                    const float2 x = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
                    part[(slot * kStGroups + g) * kStPair + a * kStTile] = x.x + x.y;
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[S_PART_FULL + slot]);
                // the pair before, which every group has left by now or soon will have
                if (due) join(pc - 1, rb);
                if (mine == 0) {
                    due = true;
                    last = j;
                    old[0] = next_old[0];
                    old[1] = next_old[1];
                }
                mine = mine == 0 ? kStGroups - 1 : mine - 1;
                ++pc;
            }
            if (due && ok) join(pc - 1, rb);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_Q_EMPTY]);
        }
    } else {
        // ------------------------------------------------------------ K
        // The warpgroups take the K tiles in turn; a thread has one token of a tile.
        regs_dec<56>();
        const int ct = tid & 127, buf = wg - 1 - kStGroups;
        constexpr int NB = D / 16;  // 16-byte pieces of the codes, read in pairs
        const int shift = p.g.page_shift, place = (1 << shift) - 1;
        const bool wide = (reinterpret_cast<uintptr_t>(p.g.kcodes) & 31u) == 0;  // 32-byte loads are aligned
        const uint32_t* table =
            reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
        const uint32_t to = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kStTmemK + (D / 2) * buf;
        // the next K tile with work after (rb, i); i = -1 starts; rb = blocks ends
        struct Step {
            int rb, i;
        };
        auto advance = [&](Step& x) {
            if (x.rb >= w.blocks) return;
            do {
                if (++x.i == w.ktiles) {
                    x.i = 0;
                    ++x.rb;
                }
            } while (x.rb < w.blocks && !w.has(x.rb, x.i));
        };
        auto entry = [&](const Step& x) {
            const int t = j0 + x.i * kStTile + ct;
            return x.rb < w.blocks && t < q.kv ? static_cast<int>(ldg_early(table + (t >> shift))) : 0;
        };
        uint4 k[NB];
        uint32_t scale;
        // pieces c, c + 1 of the row (tokens behind the end, or on a bad page, read the first token of page 0: their sums are not used)
        auto row_of = [&](const Step& x, int page) {
            const int t = j0 + x.i * kStTile + ct;
            const bool have = x.rb < w.blocks && t < q.kv && check_page(p.g, page);
            return have ? (static_cast<uint64_t>(static_cast<uint32_t>(page) * p.g.kv_heads + h) << shift) + (t & place) : 0u;
        };
        auto fetch = [&](int c, const uint8_t* src) {
            if (wide) {
                ldg_nc_32(src + 16 * c, k[c], k[c + 1]);
            } else {
                k[c] = __ldg(reinterpret_cast<const uint4*>(src + 16 * c));
                k[c + 1] = __ldg(reinterpret_cast<const uint4*>(src + 16 * c + 16));
            }
        };
        auto put = [&](int c, uint32_t f) {
            const uint32_t v[8] = {bf2_mul(codes01(k[c].x), f), bf2_mul(codes23(k[c].x), f), bf2_mul(codes01(k[c].y), f),
                                   bf2_mul(codes23(k[c].y), f), bf2_mul(codes01(k[c].z), f), bf2_mul(codes23(k[c].z), f),
                                   bf2_mul(codes01(k[c].w), f), bf2_mul(codes23(k[c].w), f)};
            tmem_st8(to + 8 * c, v);
        };
        Step now{0, -1}, next;
        for (int i = 0; i <= buf; ++i) advance(now);
        {
            const uint64_t row = row_of(now, entry(now));
#pragma unroll
            for (int c = 0; c < NB; c += 2) fetch(c, p.g.kcodes + row * D);
            scale = ldg_early(p.g.kscale + row);
        }
        next = now;
        advance(next);
        advance(next);
        int ahead = entry(next);
        bool ok = true;
        for (int n = 0; ok && now.rb < w.blocks; ++n) {
            const uint64_t row = row_of(next, ahead);
            const Step after = next;
            advance(next);
            advance(next);
            ahead = entry(next);
            ok = warp_wait(&bars[S_K_EMPTY + buf], (n & 1) ^ 1, ab, kDevTimeoutConvert);
            if (!ok) break;
            tc_fence_after();
            const uint32_t f = scale_factor(scale);
            scale = ldg_early(p.g.kscale + row);
#pragma unroll
            for (int c = 0; c < NB; c += 2) {
                put(c, f);
                put(c + 1, f);
                fetch(c, p.g.kcodes + row * D);  // the warpgroup's next tile, into the registers just freed
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_K_FULL + buf]);
            now = after;
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

template <int D, bool CAUSAL>
cudaError_t launch_d(const PagedScoreParams& p, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    constexpr uint32_t smem = StLayout<D>::kAlloc;
    static_assert(smem <= 227 * 1024, "shared memory over the sm_103 limit");
    cudaError_t e = smem_limit_once(paged_scores_tc_kernel<D, CAUSAL>, smem, configured);
    if (e != cudaSuccess) return e;
    // Ranges of cached tokens: as many blocks as fill the SMs once (a block's
    // set-up takes as long as several tiles: one sequence of 8,000 tokens x 8 KV
    // heads, 128 ranges of two tiles 15.6 us, 256 of one 22.7), at least two
    // tiles each.
    const int64_t lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    const int64_t tiles = (p.g.max_kv + kStTile - 1) / kStTile;
    const int64_t ranges = std::min<int64_t>((tiles + 1) / 2, std::max<int64_t>(1, 152 / lists));
    const int range = static_cast<int>((tiles + ranges - 1) / ranges) * kStTile;
    // (one range a list from 152 lists on: at most 65,535 x 1,024)
    const int64_t blocks = (p.g.max_kv + range - 1) / range * lists;
    paged_scores_tc_kernel<D, CAUSAL><<<static_cast<unsigned>(blocks), kStThreads, smem, s>>>(p, range);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_scores_tc(const PagedScoreParams& p, int D, cudaStream_t s) {
    if (D == 128) return p.causal ? launch_d<128, true>(p, s) : launch_d<128, false>(p, s);
    return p.causal ? launch_d<64, true>(p, s) : launch_d<64, false>(p, s);
}

}  // namespace rc
