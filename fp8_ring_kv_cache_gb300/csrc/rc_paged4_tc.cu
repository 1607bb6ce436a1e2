// rc_paged4_tc.cu -- attention of many query rows over pages of E2M1 codes, on the
// tensor cores (tcgen05).
//
// A block has up to 256 query rows of one KV head (a sequence's new tokens x
// the query heads that share it), 20 warps:
//   warp 0        issues the matrix products (one lane) and owns TMEM
//   warps 4..7    softmax group 0, warps 8..11 softmax group 1 (a row a thread)
//   warps 12..15  convert K, warps 16..19 convert V: read the codes of 128
//                 cached tokens from their pages (a tile ahead, in registers),
//                 make them fp16 and write the tile in the swizzled layout of a
//                 K-major operand, two buffers each
// A code times its block's scale is an exact fp16 number, so both products have fp16
// operands: rows of Q are brought to fp16's range by a power of two, which multiplies
// their scores in the softmax, and P has 11 bits; it is kept 2^7 larger (and the
// running maximum 7 lower), so that a weight of 2^-21 of the largest still has all of
// them.  (Scores from 2^20 on: kLargeScore4.)
// The work of a group is a chain of KV tiles: S = Q K^T into TMEM; softmax of a row by
// its thread: P to fp16, over S; O += P V with P read from TMEM.  With more than 128
// rows group i has rows [128 i, 128 i + 128) and both groups take each tile; with fewer
// both groups have the same rows and take the tiles in turn, and their results are
// joined at the end.  Either way the products of one group run while the other is in
// softmax.  P is handed over in two halves, so that the first half's products run while
// the second half's exponentials are taken, and at barriers where the softmax warps only
// arrive: the product warp looks at nothing in shared memory (a look takes 300 cycles
// beside the converters' stores), as a lane of the group has looked for it whether the
// tiles are in place.  (P handed over whole: 95 us for the chunk below; one lane that
// looks which group is ready: 119 us; units of 64 tokens with two places of scores a group,
// so that scores are always ahead: 138 us, as products of 64 columns take as long as
// those of 128.)
// 757 queries x 5,788 tokens x 48 heads x 128: 87.4 us, 1.23 PFLOP/s, 0.65 of what a
// library product of bf16 matrices reaches; the tensor cores work 52 to 55 % of the time
// of the SMs that have a block.  A tile takes 3,500 cycles for both groups, 1,750 each for
// products of 1,024.  What the rest is, is not known: by arithmetic the products' operands
// and the converters' stores are 2,048 cycles of shared memory a tile, the counters show
// its banks read in 21 % of the cycles and written in 9 % (conflicts are 3 % of the stores),
// and issue slots are used in 54 %.  A trace shows 200 to 250 cycles between the hand-over
// of a half and its products.
// A row sees the cached tokens from the first on, so a token whose V is not a number is
// remembered by the first such one's number: the row has it if it sees that far.
#include "rc_paged4.cuh"
#include "rc_paged_tc.cuh"

namespace rc {

namespace {

// The warpgroups share a launch's registers 32 + 2 x 168 + 2 x 56 = 5 x 96.

enum : int {
    F_K_FULL = 0,   // [2] the converters wrote the K tile
    F_K_EMPTY = 2,  // [2] its products have finished
    F_V_FULL = 4,
    F_V_EMPTY = 6,
    F_S_FULL = 8,   // [2] scores of group i in TMEM
    F_O_DONE = 10,
    F_DRAIN = 11,
    F_COUNT = 12
};
// Named barriers: a half of group i's P is in TMEM (the group arrives, the product warp
// waits), V's converters with the softmax groups, the two groups at the end.
constexpr int kNbHalf = 1;  // [2 groups][2 halves]
constexpr int kNbSeen = 5;
constexpr int kNbJoin = 6;
constexpr int kNbHalfThreads = 128 + 32;
constexpr int kHalfN = kTileN / 2;

template <int D>
struct Tc4Layout {
    static constexpr uint32_t kTile = kTileN * D * 2;  // bytes of an fp16 tile (Q_i, K or V)
    static constexpr uint32_t kQ = 0;                  // [2][D/64][128][128 B]
    static constexpr uint32_t kK = 2 * kTile;          // [2 buffers]
    static constexpr uint32_t kV = kK + 2 * kTile;     // [2 buffers][2 halves][D][128 B]
    static constexpr uint32_t kQScale = kV + 2 * kTile;  // what multiplies each row's scores
    static constexpr uint32_t kBar = kQScale + 4 * kRowsTc;
    static constexpr uint32_t kMisc = kBar + 8 * F_COUNT;  // [0] tmem, [1] abort, [2] first token whose V is not a number
    static constexpr uint32_t kTotal = kMisc + 64;
    static constexpr uint32_t kAlloc = kTotal + 1024;
};

// Eight bf16 numbers of a row times inv, as fp16.
__device__ __forceinline__ uint4 row_piece_f16(const uint4& w, float inv) {
    auto two = [&](uint32_t v) { return pack_f16(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xffff0000u) * inv); };
    return make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
}

// Eight codes of a word as fp16, with the factors of the pairs.
__device__ __forceinline__ uint4 scaled8(uint32_t w, uint32_t f0, uint32_t f1, uint32_t f2, uint32_t f3) {
    uint32_t r[4];
    codes8_f16(w, r);
    return make_uint4(half2_mul(r[0], f0), half2_mul(r[1], f1), half2_mul(r[2], f2), half2_mul(r[3], f3));
}

__device__ __forceinline__ uint2 ldg_early_v2(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// NUMBERED: the blocks are numbered over the tiles that there are.  (A form of its own: the sum over the lengths that finds a
// tile made the other one 1 % slower, 486 -> 491 us for 4 prompts of 259 to 2,701 new tokens.)
template <int D, bool NUMBERED>
__global__ void __launch_bounds__(kTcThreads, 1) paged4_tc_kernel(PagedAttnParams p) {
    using Lay = Tc4Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;

    // the last tiles, which see the most when causal, come first
    int b = blockIdx.x;
    const int h = b % p.g.kv_heads;
    b /= p.g.kv_heads;
    const int split = blockIdx.y;
    int s = b % p.g.seqs, tile = p.row_tiles - 1 - b / p.g.seqs;
    if constexpr (NUMBERED) {
        s = tile_place(p, b, tile, reinterpret_cast<int*>(smem));
        if (s < 0) return;
    }
    const Seq q = load_seq(p.g, s);
    const TileWork tw = tile_work(p, q, tile);
    const int row0 = tile * kRowsTc;
    if (row0 >= tw.rows || split >= tw.nsplit) return;
    const int j0 = split * p.split_tokens, j1 = min(tw.seen, j0 + p.split_tokens);
    const int rows_here = min(kRowsTc, tw.rows - row0);
    const bool two = rows_here > kTileM;              // two row tiles; else one, KV tiles in turn
    const int T = (j1 - j0 + kTileN - 1) / kTileN;    // KV tiles
    AbortState ab{reinterpret_cast<volatile uint32_t*>(&misc[1]), p.g.status, p.wait_ns};
    const int units0 = two ? T : (T + 1) / 2, units1 = two ? T : T / 2;  // tiles of a group

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[F_K_FULL + i], 4);
            mbar_init(&bars[F_K_EMPTY + i], 1);
            mbar_init(&bars[F_V_FULL + i], 4);
            mbar_init(&bars[F_V_EMPTY + i], 1);
            mbar_init(&bars[F_S_FULL + i], 1);
        }
        mbar_init(&bars[F_O_DONE], 1);
        mbar_init(&bars[F_DRAIN], 1);
        misc[1] = 0u;
        misc[2] = 0x7fffffffu;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc[0], kTcTmem);
        tmem_relinquish();
    }
    // Q rows, 8 dims a piece: kPieces lanes have a row; whole warps come here
    {
        constexpr int kPieces = D / 8;
        const int total = (two ? kRowsTc : kTileM) * kPieces;
        for (int u = tid; u < total; u += kTcThreads) {
            const int r = u / kPieces, c = u % kPieces;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (r < rows_here) {
                const int rr = row0 + r, tok = rr / p.group, head = h * p.group + rr - tok * p.group;
                w = ldg_nc_na_v4(p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D +
                                 8 * c);
            }
            float amax = 0.f;
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                amax = max3(amax, fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u)));
#pragma unroll
            for (int o = kPieces / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int e = row_exponent(amax);
            if (c == 0)
                reinterpret_cast<float*>(smem + Lay::kQScale)[r] = p.sm_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            *reinterpret_cast<uint4*>(smem + Lay::kQ + (r >> 7) * Lay::kTile + bktile_off(r & 127, 8 * c)) =
                row_piece_f16(w, __uint_as_float(static_cast<uint32_t>(127 - e) << 23));
        }
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (wg == 0) {
        regs_dec<32>();
        if (warp == 0 && T > 0) {
            // -------------------------------------------------------- products
            // Operand descriptors differ only in the start address (the low 14
            // bits, in 16 bytes; no carry below 256 KB): an add of a constant.
            constexpr uint32_t idesc_qk = instr_desc(kFmtF16, kFmtF16, 128, 128);
            constexpr uint32_t idesc_pv = instr_desc(kFmtF16, kFmtF16, 128, D);
            const uint64_t dq = smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2);
            const uint32_t hi = static_cast<uint32_t>(dq >> 32), q_lo = static_cast<uint32_t>(dq);
            const uint32_t k_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2));
            const uint32_t v_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kV), 16, 1024, 2));
            // the same in every lane, and known to be by the compiler
            const bool two_u = __shfl_sync(0xffffffffu, two ? 1 : 0, 0) != 0;
            const int n0 = __shfl_sync(0xffffffffu, units0, 0), n1 = __shfl_sync(0xffffffffu, units1, 0);
            auto issue_qk = [&](int i, int j) {
                const uint32_t d = tmem + 128u * i, qa = q_lo + ((two_u && i) ? Lay::kTile >> 4 : 0u);
                const uint32_t kb = k_lo + ((j & 1) ? Lay::kTile >> 4 : 0u);
                mma_f16_ss_at<0, 0>(d, qa, kb, hi, idesc_qk, 0);
                mma_f16_ss_at<2, 2>(d, qa, kb, hi, idesc_qk, 1);
                mma_f16_ss_at<4, 4>(d, qa, kb, hi, idesc_qk, 1);
                mma_f16_ss_at<6, 6>(d, qa, kb, hi, idesc_qk, 1);
                if (D == 128) {
                    mma_f16_ss_at<1024, 1024>(d, qa, kb, hi, idesc_qk, 1);
                    mma_f16_ss_at<1026, 1026>(d, qa, kb, hi, idesc_qk, 1);
                    mma_f16_ss_at<1028, 1028>(d, qa, kb, hi, idesc_qk, 1);
                    mma_f16_ss_at<1030, 1030>(d, qa, kb, hi, idesc_qk, 1);
                }
                mma_commit(&bars[F_S_FULL + i]);
                if (!two_u || i == 1) mma_commit(&bars[F_K_EMPTY + (j & 1)]);
            };
            auto issue_pv = [&](int i, int j, int half, bool more) {  // more: O holds something
                const uint32_t d = tmem + 256u + static_cast<uint32_t>(D) * i, pa = tmem + 128u * i + 64u * half;
                const uint32_t vb = v_lo + ((j & 1) ? Lay::kTile >> 4 : 0u) + (half ? D * 128u >> 4 : 0u);
                mma_f16_ts_at<0, 0>(d, pa, vb, hi, idesc_pv, more);
                mma_f16_ts_at<8, 2>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<16, 4>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<24, 6>(d, pa, vb, hi, idesc_pv, 1);
            };
            bool ok = true;
            const int n_all = n0 + n1;  // a group's tile each, in turn
            // the group's first scores
#pragma unroll 1
            for (int w = 0; w < 2 && w < n_all; ++w) {
                if (w == 0 || !two_u) ok = ok && warp_wait(&bars[F_K_FULL + w], 0, ab, kDevTimeoutMma);
                tc_fence_after();
                if (elect_one()) {
                    if (ok)
                        issue_qk(w, two_u ? 0 : w);
                    else
                        mbar_arrive(&bars[F_S_FULL + w]);
                }
                __syncwarp();
            }
            // Every half is waited for, also after an abort, and then the next scores are announced without products: a
            // group hands over nothing of a tile before they are, so no warp of it can be at a barrier for the second
            // time while another, or this one, has yet to come there for the first.
#pragma unroll 1
            for (int w = 0; w < n_all; ++w) {
                const int i = w & 1, j = two_u ? w >> 1 : w;
                const bool more = w + 2 < n_all;
                const uint32_t gone = *ab.flag;  // (on its way while the warp waits)
                named_barrier_sync(kNbHalf + 2 * i, kNbHalfThreads);
                ok = ok && gone == 0u;
                tc_fence_after();
                if (ok && elect_one()) issue_pv(i, j, 0, w > 1);
                __syncwarp();
                named_barrier_sync(kNbHalf + 2 * i + 1, kNbHalfThreads);
                tc_fence_after();
                if (elect_one()) {
                    if (ok) {
                        issue_pv(i, j, 1, true);
                        if (!two_u || i == 1) mma_commit(&bars[F_V_EMPTY + (j & 1)]);
                        if (more) issue_qk(i, two_u ? j + 1 : j + 2);
                    } else if (more) {
                        mbar_arrive(&bars[F_S_FULL + i]);
                    }
                }
                __syncwarp();
            }
            if (elect_one()) {  // (the lane that issued the products commits them)
                if (ok) mma_commit(&bars[F_O_DONE]);
                // every product has finished before the tensor memory is released
                mma_commit(&bars[F_DRAIN]);
            }
            __syncwarp();
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars[F_DRAIN], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else if (wg < kWgConvertK) {
        // ------------------------------------------------------------ softmax
        regs_inc<168>();
        const int i = wg - kWgSoftmax0;
        const int quad = warp & 3, r = quad * 32 + lane;  // TMEM lane quadrant; row within the group's tile
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t s_tm = tmem + lane_off + 128u * i;
        const uint32_t o_tm = tmem + lane_off + 256u + static_cast<uint32_t>(D) * i;
        const int rr = row0 + (two ? kTileM * i : 0) + r;  // row of the KV head
        const bool live = rr < tw.rows;
        const int tok = live ? rr / p.group : 0, head = h * p.group + (live ? rr - tok * p.group : 0);
        // tokens the row sees, counted from j0; rows past the end see all (nothing of theirs is stored)
        const int limit = (!live || !p.causal ? j1 : min(j1, max(0, q.kv - q.n + tok + 1))) - j0;
        const float a = reinterpret_cast<const float*>(smem + Lay::kQScale)[(two ? kTileM * i : 0) + r];
        const float2 a2 = make_float2(a, a);
        const bool may_be_large = __any_sync(0xffffffffu, live && a >= p.sm_log2 * kLargeQuery4);
        constexpr float kBelow = 7.f;  // of the running maximum
        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        const int units = i ? units1 : units0;
        const bool watcher = quad == 0 && lane == 0;
        auto hand_over = [&](int half) {
            tc_fence_before();
            __syncwarp();
            named_barrier_arrive(kNbHalf + 2 * i + half, kNbHalfThreads);
        };
#pragma unroll 1
        for (int u = 0; u < units; ++u) {
            const int j = two ? u : 2 * u + i;
            if (ok) ok = warp_wait(&bars[F_S_FULL + i], u & 1, ab, kDevTimeoutSoftmax);
            if (!ok) {
                // after an abort: the halves are handed over still, and not before their turn, which the scores announce
                // (the product warp always comes to that; the bound is for what nobody thought of)
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(&bars[F_S_FULL + i], u & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
                }
                hand_over(0);
                hand_over(1);
                continue;
            }
            // V of this tile and K of the group's next, tested now and looked at after the exponentials.  (Not before the
            // scores are there: a buffer's phase before the last would pass for the one that is wanted.)
            const int jk = two ? j + 1 : j + 2;
            bool v_in = true, k_in = true;
            if (watcher) {
                v_in = mbar_test(&bars[F_V_FULL + (j & 1)], (j >> 1) & 1);
                if (u + 1 < units) k_in = mbar_test(&bars[F_K_FULL + (jk & 1)], (jk >> 1) & 1);
            }
            tc_fence_after();
            const int room = limit - j * kTileN;  // columns the row sees
            uint32_t x[kTileN];
            tmem_ld128(s_tm, x);
            if (!__all_sync(0xffffffffu, room >= kTileN)) {
#pragma unroll
                for (int k = 0; k < kTileN; ++k)
                    if (k >= room) x[k] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mx[c] = fmaxf(__uint_as_float(x[c]), __uint_as_float(x[4 + c]));
#pragma unroll
                for (int k = 8; k < kTileN; k += 8)
                    mx[c] = max3(mx[c], __uint_as_float(x[k + c]), __uint_as_float(x[k + 4 + c]));
            }
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float m_tile = fmaf(most, a, -kBelow);
            // the running max moves only when a tile raises it by more than 2^8 of
            // weight: fp16 (up to 2^15) and fp32 hold the larger weights as well
            const bool bump = (m_run == -INFINITY) || (m_tile > m_run + 8.f);
            float m_new = bump ? fmaxf(m_run, m_tile) : m_run;
            float base = (m_new == -INFINITY) ? 0.f : m_new;
            float alpha = bump ? ex2(m_run - base) : 1.f;
            // rescale the running output when the max moved (the products of the tile before have finished: the scores
            // came after them)
            auto rescale = [&](float by) {
                if (!__any_sync(0xffffffffu, u > 0 && by != 1.f)) return;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t y[16];
                    tmem_ld16(o_tm + 16 * c, y);
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * by);
                    tmem_st16(o_tm + 16 * c, y);
                }
                tmem_st_wait();
            };
            rescale(alpha);
            float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
            auto give = [&](int half) {
                tmem_st_wait();
                if (watcher && half == 0 && !v_in) ok = mbar_wait(&bars[F_V_FULL + (j & 1)], (j >> 1) & 1, ab, kDevTimeoutSoftmax);
                if (watcher && half == 1 && !k_in) ok = mbar_wait(&bars[F_K_FULL + (jk & 1)], (jk >> 1) & 1, ab, kDevTimeoutSoftmax) && ok;
                hand_over(half);
            };
            if (may_be_large && __any_sync(0xffffffffu, fabsf(base) >= kLargeScore4)) {
                if (fabsf(base) >= kLargeScore4) m_new = fmaxf(base, __fmul_rn(most, a));
                const float by = m_new == -INFINITY ? 1.f : ex2(base - m_new);
                rescale(by);
                alpha *= by;
                base = m_new == -INFINITY ? 0.f : m_new;
                // (a few columns at a time, so that this costs the other way no registers)
#pragma unroll 1
                for (int c = 0; c < kTileN / 32; ++c) {
                    uint32_t y[32], pk[16];
                    tmem_ld32(s_tm + 32 * c, y);
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float2 w;
                        w.x = ex2(32 * c + k < room ? __fadd_rn(__fmul_rn(__uint_as_float(y[k]), a), -base) : -INFINITY);
                        w.y = ex2(32 * c + k + 1 < room ? __fadd_rn(__fmul_rn(__uint_as_float(y[k + 1]), a), -base) : -INFINITY);
                        ls0 = add2(ls0, w);
                        pk[k / 2] = pack_f16(w.x, w.y);
                    }
                    tmem_st16(s_tm + 16 * (c & 1) + kHalfN * (c >> 1), pk);
                    if (c & 1) give(c >> 1);
                }
            } else {
                const float2 n2 = make_float2(-base, -base);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int k = 0; k < kHalfN; k += 4) {
                        const uint32_t* w = x + kHalfN * half + k;
                        const float2 x0 = fma2(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), a2, n2);
                        const float2 x1 = fma2(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), a2, n2);
                        const float2 q0 = make_float2(ex2(x0.x), ex2(x0.y));
                        const float2 q1 = make_float2(ex2(x1.x), ex2(x1.y));
                        ls0 = add2(ls0, q0);
                        ls1 = add2(ls1, q1);
                        pk[k / 2] = pack_f16(q0.x, q0.y);
                        pk[k / 2 + 1] = pack_f16(q1.x, q1.y);
                    }
                    tmem_st32(s_tm + kHalfN * half, pk);
                    give(half);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            l_run = l_run * alpha + ((ls0.x + ls0.y) + (ls1.x + ls1.y));
            m_run = m_new;
        }
        // ------------------------------------------------------------ epilogue
        named_barrier_sync(kNbSeen, 128 + 256);
        bool poison = static_cast<int>(misc[2]) < limit;  // a token whose V is not a number is seen
        if (ok && T > 0) ok = warp_wait(&bars[F_O_DONE], 0, ab, kDevTimeoutEpilogue);
        tc_fence_after();
        // With one row tile the groups' results are joined: group 1 leaves its
        // max, sum and O in shared memory (the K and V buffers, free once every
        // product has finished).
        float scale = 1.f, other = 0.f;
        const float* theirs = reinterpret_cast<const float*>(smem + Lay::kK) + quad * 32 * 36;
        if (!two) {
            float* ml = reinterpret_cast<float*>(smem + Lay::kV + Lay::kTile);  // [128] max, [128] sum
            if (i == 1) {
                ml[r] = m_run;
                ml[128 + r] = l_run;
                if (units1 > 0 && ok) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t y[32];
                        tmem_ld32(o_tm + 32 * c, y);
                        float* dst = reinterpret_cast<float*>(smem + Lay::kK) + c * (128 * 36) + quad * 32 * 36 + lane * 36;
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4*>(dst + k) = make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    }
                }
            }
            ok = named_barrier_and(kNbJoin, 256, ok);
            if (i == 0) {
                const float m1 = ml[r], l1 = ml[128 + r];
                const float M = fmaxf(m_run, m1);
                scale = m_run == -INFINITY ? 0.f : ex2(m_run - M);
                other = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                l_run = l_run * scale + l1 * other;
                m_run = M;
            }
        }
        if (ok && (two || i == 0)) {
            const bool last = tw.nsplit == 1;
            const float inv = !last ? 1.f : (l_run > 0.f || l_run != l_run) ? 1.f / l_run : 0.f;
            const float f = poison ? __uint_as_float(0x7fc00000u) : scale * inv;
            const float g = other * inv;
            const int slot = (s * p.row_tiles + tile) * p.g.kv_heads + h;
            float* part = p.part + (static_cast<size_t>(slot) * p.splits + split) * tc_part_floats<D>();
            const int tr = (two ? kTileM * i : 0) + r;  // row of the 256
            if (live) {
                if (!last) {
                    part[kRowsTc * D + tr] = m_run;
                    part[kRowsTc * D + kRowsTc + tr] = l_run;
                } else if (p.lse != nullptr) {
                    p.lse[static_cast<int64_t>(q.q0 + tok) * p.heads + head] =
                        l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
                }
            }
            // Rows go out through shared memory (the Q image, which no product
            // reads any more), so that a store instruction covers whole lines.
            float* stage = reinterpret_cast<float*>(smem + Lay::kQ) + (i * 4 + quad) * (32 * 36);
            const int wrow = row0 + (two ? kTileM * i : 0) + quad * 32;  // the warp's first row
            const bool both = !two && units1 > 0;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t y[32];
                if (T > 0) tmem_ld32(o_tm + 32 * c, y);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (T > 0)
                        x = make_float4(__uint_as_float(y[k]) * f, __uint_as_float(y[k + 1]) * f,
                                        __uint_as_float(y[k + 2]) * f, __uint_as_float(y[k + 3]) * f);
                    if (both) {
                        const float4 z = *reinterpret_cast<const float4*>(theirs + c * (128 * 36) + lane * 36 + k);
                        x = make_float4(fmaf(z.x, g, x.x), fmaf(z.y, g, x.y), fmaf(z.z, g, x.z), fmaf(z.w, g, x.w));
                    }
                    *reinterpret_cast<float4*>(stage + lane * 36 + k) = x;
                }
                __syncwarp();
                if (last) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int ro = 8 * k + (lane >> 2), e = 8 * (lane & 3);
                        const int row = wrow + ro;
                        const float4 x = *reinterpret_cast<const float4*>(stage + ro * 36 + e);
                        const float4 z = *reinterpret_cast<const float4*>(stage + ro * 36 + e + 4);
                        if (row < tw.rows) {
                            const int t2 = row / p.group, h2 = h * p.group + row - t2 * p.group;
                            *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(q.q0 + t2) * p.out_stride +
                                                      static_cast<int64_t>(h2) * D + 32 * c + e) =
                                make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(z.x, z.y),
                                           pack_bf16(z.z, z.w));
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int ro = 4 * k + (lane >> 3), e = 4 * (lane & 7);
                        if (wrow + ro < tw.rows)
                            *reinterpret_cast<float4*>(part + static_cast<size_t>(wrow + ro - row0) * D + 32 * c + e) =
                                *reinterpret_cast<const float4*>(stage + ro * 36 + e);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------ converters
        // Warpgroup 3 converts K, warpgroup 4 V, each its next tile in registers
        // while it waits for a free buffer.  Lane l < 8 of a warp looks up where
        // the tile's tokens [16 l, 16 l + 16) are: the number of their block of
        // 16 among the pool's (page, head, 16 tokens).  Blocks behind the end of
        // the sequence, or on a bad page, read block 0 instead.  Behind the end the
        // softmax cuts K's columns, and V's get the scale 0, as P is 0 there; a bad
        // page's tokens have block 0's scores and V, and the call's results are void.
        regs_dec<56>();
        const int ct = tid & 127;
        const int pb = p.g.page_shift - 4;  // blocks of a page: 1 << pb
        bool ok = true;
        const uint32_t* table =
            reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
        // the page table's entry is read two tiles ahead and looked at one
        // tile ahead, so no load waits for another
        auto entry_at = [&](int j) {
            const int t = j0 + j * kTileN + 16 * (lane & 7);
            return j < T && t < q.kv ? static_cast<int>(ldg_early(table + (t >> p.g.page_shift))) : 0;
        };
        auto block_of = [&](int j, int page) {
            const int t = j0 + j * kTileN + 16 * (lane & 7);
            if (j >= T || t >= q.kv) return 0u;
            const uint32_t at = static_cast<uint32_t>(check_page(p.g, page) ? page : 0) * p.g.kv_heads + h;
            return (at << pb) + (static_cast<uint32_t>(t >> 4) & ((1u << pb) - 1u));
        };
        auto place = [&](uint32_t at) { return 16 * (at & ((1u << pb) - 1u)); };  // of a block in its page
        int ahead = entry_at(1);
        if (wg == kWgConvertK) {
            // rows rr + 32 m, dims D / 4 (ct % 4) ..: KW words of eight codes, in 16-byte pieces of the tile.  The lanes
            // of the second 64 dims (D = 128) take the pieces in the order 2, 3, 0, 1: eight lanes' stores then meet no
            // bank conflict.
            constexpr int KW = D / 32, KB = D / 64;
            struct Ahead {
                uint32_t codes[4][KW], scales[4][KB];
            };
            const int rr = ct >> 2, qd = ct & 3;
            const bool swap = D == 128 && (qd & 2);
            const uint8_t* kbase = p.g.kcodes + (rr & 15) * (D / 2) + qd * (D / 8);
            const uint8_t* sbase = p.g.kscale + ((KB * qd) << p.g.page_shift) + (rr & 15);
            auto fetch = [&](Ahead& to, int m, uint32_t blk) {
                const uint32_t at = __shfl_sync(0xffffffffu, blk, (rr >> 4) + 2 * m);
                const uint8_t* from = kbase + static_cast<uint64_t>(at) * (16 * D / 2);
                if constexpr (KW == 4) {
                    const uint4 w = ldg_nc_na_v4(from);
                    to.codes[m][0] = w.x, to.codes[m][1] = w.y, to.codes[m][2] = w.z, to.codes[m][3] = w.w;
                } else {
                    const uint2 w = ldg_early_v2(from);
                    to.codes[m][0] = w.x, to.codes[m][1] = w.y;
                }
                const uint8_t* sc = sbase + ((static_cast<uint64_t>(at >> pb) * (D / 16)) << p.g.page_shift) + place(at);
#pragma unroll
                for (int n = 0; n < KB; ++n) to.scales[m][n] = ldg_early(sc + (n << p.g.page_shift));
            };
            const uint32_t off = bktile_off(rr, (D / 4) * qd + (swap ? 16 : 0));
            auto convert = [&](Ahead& a, int j) {
                const uint32_t blk = block_of(j + 1, ahead);  // (block 0 past the last tile: read, not used)
                ahead = entry_at(j + 2);
                ok = warp_wait(&bars[F_K_EMPTY + (j & 1)], ((j >> 1) & 1) ^ 1, ab, kDevTimeoutConvert);
                if (!ok) return;
                uint8_t* dst = smem + Lay::kK + (j & 1) * Lay::kTile;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t w[KW], f[KB];
#pragma unroll
                    for (int k = 0; k < KW; ++k) w[k] = swap ? a.codes[m][k ^ (KW == 4 ? 2 : 0)] : a.codes[m][k];
#pragma unroll
                    for (int n = 0; n < KB; ++n) f[n] = (swap ? a.scales[m][n ^ (KB - 1)] : a.scales[m][n]) * 0x00800080u;
#pragma unroll
                    for (int k = 0; k < KW; ++k)
                        *reinterpret_cast<uint4*>(dst + (off ^ (16u * k)) + m * (32 * 128)) =
                            scaled8(w[k], f[k / 2], f[k / 2], f[k / 2], f[k / 2]);
                    fetch(a, m, blk);  // the next tile's rows, into the registers just freed
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[F_K_FULL + (j & 1)]);
            };
            Ahead a0;
            if (T > 0) {
                const uint32_t b0 = block_of(0, entry_at(0));
#pragma unroll
                for (int m = 0; m < 4; ++m) fetch(a0, m, b0);
            }
#pragma unroll 1
            for (int j = 0; ok && j < T; ++j) convert(a0, j);
        } else {
            // tokens 16 c .. of the dims 16 nb + dd + DS k, which have one scale a token
            constexpr int VU = D / 16, DS = 16 / VU;
            struct Ahead {
                uint2 codes[VU];
                uint4 scales;
            };
            const int c = (ct & 3) | ((ct >> 4) & 4), dd = (ct >> 2) & (DS - 1), nb = (ct / (4 * DS)) & (D / 16 - 1);
            const int d0 = 16 * nb + dd;
            const uint32_t step = static_cast<uint32_t>(DS) << (p.g.page_shift - 1);  // DS dims
            auto source = [&](uint32_t at) {
                return p.g.vcodes + (((static_cast<uint64_t>(at >> pb) * D + d0) << p.g.page_shift) + place(at)) / 2;
            };
            auto scales_at = [&](uint32_t at) {
                return ldg_nc_na_v4(p.g.vscale + ((static_cast<uint64_t>(at >> pb) * (D / 16) + nb) << p.g.page_shift) + place(at));
            };
            auto convert = [&](Ahead& a, int j) {
                const uint32_t at = __shfl_sync(0xffffffffu, block_of(j + 1, ahead), c);
                ahead = entry_at(j + 2);
                ok = warp_wait(&bars[F_V_EMPTY + (j & 1)], ((j >> 1) & 1) ^ 1, ab, kDevTimeoutConvert);
                if (!ok) return;
                const int first = j0 + j * kTileN + 16 * c;  // token
                const uint4 cut = cut16(a.scales, q.kv - first);
                uint32_t w[4] = {cut.x, cut.y, cut.z, cut.w};
                if ((nan_scales(w[0]) | nan_scales(w[1]) | nan_scales(w[2]) | nan_scales(w[3])) != 0u) {
                    // a V that is not a number counts as 0 in the product; the first 16 dims' scale says that the token is one
                    int bad_at = 16;
#pragma unroll
                    for (int k = 3; k >= 0; --k) {
                        const uint32_t bad = nan_scales(w[k]);
                        if (bad) bad_at = 4 * k + ((__ffs(bad) - 1) >> 3);
                        w[k] &= ~((bad >> 7) * 0xffu);
                    }
                    if (nb == 0) atomicMin(reinterpret_cast<int*>(&misc[2]), first - j0 + bad_at);
                }
                uint32_t f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = scales01(w[k]);
                    f[2 * k + 1] = scales23(w[k]);
                }
                a.scales = scales_at(at);
                const uint8_t* src = source(at);
                uint8_t* dst = smem + Lay::kV + (j & 1) * Lay::kTile;
#pragma unroll
                for (int k = 0; k < VU; ++k) {
                    // (eight lanes: four blocks of tokens, two neighbouring dims, whose swizzles differ in the lowest bit)
                    const int d = d0 + DS * k;
                    *reinterpret_cast<uint4*>(dst + bvtile_off(d, 16 * c, D)) = scaled8(a.codes[k].x, f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4*>(dst + bvtile_off(d, 16 * c + 8, D)) = scaled8(a.codes[k].y, f[4], f[5], f[6], f[7]);
                    a.codes[k] = ldg_early_v2(src + k * step);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[F_V_FULL + (j & 1)]);
            };
            Ahead a0;
            if (T > 0) {
                const uint32_t at0 = __shfl_sync(0xffffffffu, block_of(0, entry_at(0)), c);
#pragma unroll
                for (int k = 0; k < VU; ++k) a0.codes[k] = ldg_early_v2(source(at0) + k * step);
                a0.scales = scales_at(at0);
            }
#pragma unroll 1
            for (int j = 0; ok && j < T; ++j) convert(a0, j);
            named_barrier_sync(kNbSeen, 128 + 256);  // (also after an abort: the softmax groups come there)
        }
    }

    // ------------------------------------------------------------ teardown
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTcTmem);
    }
}

template <int D>
cudaError_t launch_d(PagedAttnParams& p, size_t part_floats_max, cudaStream_t s) {
    static std::atomic<uint64_t> configured[2]{};
    constexpr uint32_t smem = Tc4Layout<D>::kAlloc;
    static_assert(smem <= 227 * 1024, "shared memory over the sm_103 limit");
    return launch_tiles<D>({paged4_tc_kernel<D, false>, configured[0]}, {paged4_tc_kernel<D, true>, configured[1]}, smem, p, part_floats_max, s);
}

}  // namespace

cudaError_t launch_paged4_tc(PagedAttnParams& p, int D, size_t part_floats_max, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, part_floats_max, s) : launch_d<64>(p, part_floats_max, s);
}

}  // namespace rc
