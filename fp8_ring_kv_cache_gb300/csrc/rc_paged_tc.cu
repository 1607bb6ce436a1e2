// rc_paged_tc.cu -- attention of many query rows over the pages, on the
// tensor cores (tcgen05).
//
// A block has up to 256 query rows of one KV head (a sequence's new tokens x
// the query heads that share it), 20 warps:
//   warp 0        issues the matrix products (one lane) and owns TMEM
//   warps 4..7    softmax group 0, warps 8..11 softmax group 1 (a row a thread)
//   warps 12..15  convert K, warps 16..19 convert V: read the codes of 128
//                 cached tokens from their pages (a tile ahead, in registers),
//                 make them bf16 and write the tile in the swizzled layout of a
//                 K-major operand, two buffers each
// Scales are powers of two, so the bf16 tiles are exact, S = Q K^T needs no
// factor per column, and both products run at the bf16 rate:
//   S_i = Q_i K_j^T into TMEM; softmax of a row by its thread: P to bf16, over
//   S in TMEM; O_i += P_i V_j with P read from TMEM.
// The work is a chain of units: unit u is (KV tile, group u & 1).  With more
// than 128 rows group i has rows [128 i, 128 i + 128) and both groups take
// each KV tile; with fewer both groups have the same rows and take the KV tiles
// in turn, and their results are joined at the end.  Either way the products of
// one group run while the other is in softmax.  After P of unit u: O += P V of
// unit u, then S of unit u + 2, which overwrites P's place.
// P is rounded to bf16 (its row sums are not): the operands of a product are of one
// type, and V's values, exact in bf16, need its range (2^-133 to 57,344), so P cannot
// have fp16's 11 bits, which the 16-bit ring's attention gives it.  Two bf16 parts of
// P would hold 16 bits of it for half as many products again.  The rounding of P adds
// to that of the bf16 result: an error of 0.0020 (the chunk below) and 0.0021 (ragged
// prompts) of the result's norm, where the bf16 result alone has 0.0017.
// A code word gives the pairs (0, 2) and (1, 3) of its four values cheapest:
// that order is kept along the summed dims (Q is stored in it) and along the
// cached tokens (P is packed in it).
//
// 757 queries x 5,788 tokens x 48 heads x 128: 102 us, 1.05 PFLOP/s, 0.56 of what
// a library product of bf16 matrices reaches; the tensor cores work 47 % of the
// time.  What bounds it is the chain of a unit (scores to registers, maximum,
// exponentials, P back, the hand-over to the products), which two groups do not
// quite hide; the converters of K keep up just so (the marks of V rows that are
// not numbers, some 40 instructions a tile, cost 2 us while one of them made them).
#include "rc_paged_tc.cuh"

namespace rc {

namespace {

// The warpgroups share a launch's registers 32 + 2 x 168 + 2 x 56 = 5 x 96.

enum : int {
    T_K_FULL = 0,   // [2] the converters wrote the K tile
    T_K_EMPTY = 2,  // [2] its products have finished
    T_V_FULL = 4,
    T_V_EMPTY = 6,
    T_S_FULL = 8,  // [2] scores of group i in TMEM
    T_O_DONE = 10,
    T_DRAIN = 11,
    T_COUNT = 12
};
// Named barriers: group i with the product warp (P in TMEM; the group's
// watching lane has seen V of this unit and K of unit u + 2), and the two
// groups at the end.
constexpr int kNbUnit = 1;  // [2]
constexpr int kNbJoin = 3;
constexpr int kNbUnitThreads = 128 + 32;

template <int D>
struct TcLayout {
    static constexpr uint32_t kTile = kTileN * D * 2;  // bytes of a bf16 tile (Q_i, K or V)
    static constexpr uint32_t kQ = 0;                  // [2][D/64][128][128 B]
    static constexpr uint32_t kK = 2 * kTile;          // [2 buffers]
    static constexpr uint32_t kV = kK + 2 * kTile;     // [2 buffers][2 halves][D][128 B]
    static constexpr uint32_t kScale = kV + 2 * kTile; // V scale bytes of the last four KV tiles
    static constexpr uint32_t kBar = kScale + 4 * kTileN;
    static constexpr uint32_t kMisc = kBar + 8 * T_COUNT;  // [0] tmem, [1] abort, [4..11] half of a KV tile holds a V that is not a number
    static constexpr uint32_t kTotal = kMisc + 64;
    static constexpr uint32_t kAlloc = kTotal + 1024;
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) paged_tc_kernel(PagedAttnParams p) {
    using Lay = TcLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;

    // the last tiles, which see the most when causal, come first
    int b = blockIdx.x;
    const int h = b % p.g.kv_heads;
    b /= p.g.kv_heads;
    const int s = b % p.g.seqs, tile = p.row_tiles - 1 - b / p.g.seqs, split = blockIdx.y;
    const Seq q = load_seq(p.g, s);
    const TileWork tw = tile_work(p, q, tile);
    const int row0 = tile * kRowsTc;
    if (row0 >= tw.rows || split >= tw.nsplit) return;
    const int j0 = split * p.split_tokens, j1 = min(tw.seen, j0 + p.split_tokens);
    const int rows_here = min(kRowsTc, tw.rows - row0);
    const bool two = rows_here > kTileM;              // two row tiles; else one, KV tiles in turn
    const int T = (j1 - j0 + kTileN - 1) / kTileN;    // KV tiles
    const int U = two ? 2 * T : T;                    // units
    AbortState ab{reinterpret_cast<volatile uint32_t*>(&misc[1]), p.g.status, p.wait_ns};
    auto tile_of = [&](int u) { return two ? u >> 1 : u; };

    // ------------------------------------------------------------ set-up
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[T_K_FULL + i], 4);
            mbar_init(&bars[T_K_EMPTY + i], 1);
            mbar_init(&bars[T_V_FULL + i], 4);
            mbar_init(&bars[T_V_EMPTY + i], 1);
            mbar_init(&bars[T_S_FULL + i], 1);
        }
        mbar_init(&bars[T_O_DONE], 1);
        mbar_init(&bars[T_DRAIN], 1);
        misc[1] = 0u;
        for (int i = 4; i < 12; ++i) misc[i] = 0u;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&misc[0], kTcTmem);
        tmem_relinquish();
    }
    // Q rows, 8 dims a piece, in the order (0, 2), (1, 3) of each four
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
            *reinterpret_cast<uint4*>(smem + Lay::kQ + (r >> 7) * Lay::kTile + bktile_off(r & 127, 8 * c)) =
                make_uint4(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632),
                           __byte_perm(w.z, w.w, 0x5410), __byte_perm(w.z, w.w, 0x7632));
        }
        fence_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];

    if (wg == 0) {
        regs_dec<32>();
        if (warp == 0 && U > 0) {
            // -------------------------------------------------------- products
            // Operand descriptors differ only in the start address (the low 14
            // bits, in 16 bytes; no carry below 256 KB): an add of a constant.
            const uint32_t idesc_qk = instr_desc(kFmtBF16, kFmtBF16, 128, 128);
            const uint32_t idesc_pv = instr_desc(kFmtBF16, kFmtBF16, 128, D);
            const uint64_t dq = smem_desc(smem_u32(smem + Lay::kQ), 16, 1024, 2);
            const uint32_t hi = static_cast<uint32_t>(dq >> 32), q_lo = static_cast<uint32_t>(dq);
            const uint32_t k_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kK), 16, 1024, 2));
            const uint32_t v_lo = static_cast<uint32_t>(smem_desc(smem_u32(smem + Lay::kV), 16, 1024, 2));
            // the same in every lane, and known to be by the compiler
            const bool two_u = __shfl_sync(0xffffffffu, two ? 1 : 0, 0) != 0;
            const int U_u = __shfl_sync(0xffffffffu, U, 0);
            auto issue_qk = [&](int u) {
                const int i = u & 1, j = two_u ? u >> 1 : u;
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
                mma_commit(&bars[T_S_FULL + i]);
                if (!two_u || i == 1) mma_commit(&bars[T_K_EMPTY + (j & 1)]);
            };
            auto issue_pv = [&](int u) {
                const int i = u & 1, j = two_u ? u >> 1 : u;
                const uint32_t d = tmem + 256u + static_cast<uint32_t>(D) * i, pa = tmem + 128u * i;
                const uint32_t vb = v_lo + ((j & 1) ? Lay::kTile >> 4 : 0u);
                constexpr uint32_t H = D * 128 / 16;  // the second 64 tokens
                mma_f16_ts_at<0, 0>(d, pa, vb, hi, idesc_pv, u > 1);
                mma_f16_ts_at<8, 2>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<16, 4>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<24, 6>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<32, H>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<40, H + 2>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<48, H + 4>(d, pa, vb, hi, idesc_pv, 1);
                mma_f16_ts_at<56, H + 6>(d, pa, vb, hi, idesc_pv, 1);
                if (!two_u || i == 1) mma_commit(&bars[T_V_EMPTY + (j & 1)]);
            };
            bool ok = true;
#pragma unroll 1
            for (int u = 0; u < 2 && u < U_u; ++u) {
                ok = ok && warp_wait(&bars[T_K_FULL + ((two_u ? 0 : u) & 1)], 0, ab, kDevTimeoutMma);
                tc_fence_after();
                if (ok && elect_one()) issue_qk(u);
                __syncwarp();
            }
            // every unit passes its rendezvous, also after an abort, so no partner is left waiting
#pragma unroll 1
            for (int u = 0; u < U_u; ++u) {
                ok = named_barrier_and(kNbUnit + (u & 1), kNbUnitThreads, ok);
                tc_fence_after();
                if (ok && elect_one()) {
                    issue_pv(u);
                    if (u + 2 < U_u) issue_qk(u + 2);
                }
                __syncwarp();
            }
            // (the lane that issued the products commits them)
            if (elect_one()) {
                if (ok) mma_commit(&bars[T_O_DONE]);
                // every product has finished before the tensor memory is released
                mma_commit(&bars[T_DRAIN]);
            }
            __syncwarp();
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars[T_DRAIN], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
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
        const float a = p.sm_log2;
        const float2 a2 = make_float2(a, a);
        float m_run = -INFINITY, l_run = 0.f;
        bool poison = false;  // a token whose V is not a number is seen
        bool ok = true;
        const bool watcher = quad == 0 && lane == 0;

        // whether the row sees a token of the unit's tile whose V is not a number (once its V is known to be in place)
        auto look = [&](int u) {
            const int j = tile_of(u);
            if ((misc[4 + (j & 3)] | misc[8 + (j & 3)]) == 0u) return;
            const uint8_t* vs = smem + Lay::kScale + (j & 3) * kTileN;
            for (int k = 0; k < kTileN; ++k) poison |= vs[k] > 134 && k < limit - j * kTileN;
        };

        auto unit = [&](int u) -> bool {
            const int j = tile_of(u);
            if (!warp_wait(&bars[T_S_FULL + i], (u >> 1) & 1, ab, kDevTimeoutSoftmax)) return false;
            // V of this unit and K of unit u + 2, tested now and looked at after the softmax.  (Not before the scores are
            // there: with one row tile K of unit u lies in the same buffer, and while it is not in place the test would
            // answer for the phase before.  Nor is it faster, where it can be done: 104.1 us for the chunk above.)
            const int jk = tile_of(u + 2);
            const bool want_k = u + 2 < U;
            bool vk = true;
            if (watcher) {
                vk = mbar_test(&bars[T_V_FULL + (j & 1)], (j >> 1) & 1);
                if (want_k) vk = mbar_test(&bars[T_K_FULL + (jk & 1)], (jk >> 1) & 1) && vk;
            }
            tc_fence_after();
            const int room = limit - j * kTileN;  // columns the row sees
            uint32_t v[128];
            tmem_ld128(s_tm, v);
            if (!__all_sync(0xffffffffu, room >= kTileN)) {
#pragma unroll
                for (int k = 0; k < kTileN; ++k)
                    if (k >= room) v[k] = 0xff800000u;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mx[c] = fmaxf(__uint_as_float(v[c]), __uint_as_float(v[4 + c]));
#pragma unroll
                for (int k = 8; k < kTileN; k += 8)
                    mx[c] = max3(mx[c], __uint_as_float(v[k + c]), __uint_as_float(v[k + 4 + c]));
            }
            const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a;
            // the running max moves only when a tile raises it by more than
            // 2^8 of weight: bf16 and fp32 hold the larger weights as well
            const bool bump = (m_run == -INFINITY) || (m_tile > m_run + 8.f);
            const float m_new = bump ? fmaxf(m_run, m_tile) : m_run;
            const float base = (m_new == -INFINITY) ? 0.f : m_new;
            const float alpha = bump ? ex2(m_run - base) : 1.f;
            const float2 n2 = make_float2(-base, -base);
            float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 64; k += 4) {
                    const uint32_t* w = v + 64 * half + k;
                    const float2 x0 = fma2(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), a2, n2);
                    const float2 x1 = fma2(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), a2, n2);
                    const float2 q0 = make_float2(ex2(x0.x), ex2(x0.y));
                    const float2 q1 = make_float2(ex2(x1.x), ex2(x1.y));
                    ls0 = add2(ls0, q0);
                    ls1 = add2(ls1, q1);
                    pk[k / 2] = pack_bf16(q0.x, q1.x);      // tokens 0, 2
                    pk[k / 2 + 1] = pack_bf16(q0.y, q1.y);  // tokens 1, 3
                }
                tmem_st32(s_tm + 32 * half, pk);
            }
            tmem_st_wait();
            // rescale the running output when the max moved (the product of
            // unit u - 2 has finished: S of this unit came after it)
            if (__any_sync(0xffffffffu, u > 1 && alpha != 1.f)) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(o_tm + 32 * c, v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                    tmem_st32(o_tm + 32 * c, v);
                }
                tmem_st_wait();
            }
            l_run = l_run * alpha + ((ls0.x + ls0.y) + (ls1.x + ls1.y));
            m_run = m_new;
            if (watcher && !vk) {
                if (!mbar_wait(&bars[T_V_FULL + (j & 1)], (j >> 1) & 1, ab, kDevTimeoutSoftmax)) return false;
                if (want_k && !mbar_wait(&bars[T_K_FULL + (jk & 1)], (jk >> 1) & 1, ab, kDevTimeoutSoftmax)) return false;
            }
            return true;
        };
        for (int u = i; u < U; u += 2) {
            if (ok) ok = unit(u);
            tc_fence_before();
            __syncwarp();
            ok = named_barrier_and(kNbUnit + i, kNbUnitThreads, ok);
            if (ok) look(u);
        }
        // ------------------------------------------------------------ epilogue
        if (ok && U > 0) ok = warp_wait(&bars[T_O_DONE], 0, ab, kDevTimeoutEpilogue);
        tc_fence_after();
        // With one row tile the groups' results are joined: group 1 leaves its
        // max, sum and O in shared memory (the K and V buffers, free once every
        // product has finished).
        float scale = 1.f, other = 0.f;
        const float* theirs = reinterpret_cast<const float*>(smem + Lay::kK) + quad * 32 * 36;
        if (!two) {
            float* ml = reinterpret_cast<float*>(smem + Lay::kV + Lay::kTile);  // [128] max, [128] sum, [128] poison
            if (i == 1) {
                ml[r] = m_run;
                ml[128 + r] = l_run;
                ml[256 + r] = poison ? 1.f : 0.f;
                if (U > 1 && ok) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(o_tm + 32 * c, v);
                        float* dst = reinterpret_cast<float*>(smem + Lay::kK) + c * (128 * 36) + quad * 32 * 36 + lane * 36;
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<uint4*>(dst + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
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
                poison |= ml[256 + r] != 0.f;
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
            const bool both = !two && U > 1;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                if (U > 0) tmem_ld32(o_tm + 32 * c, v);
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (U > 0)
                        x = make_float4(__uint_as_float(v[k]) * f, __uint_as_float(v[k + 1]) * f,
                                        __uint_as_float(v[k + 2]) * f, __uint_as_float(v[k + 3]) * f);
                    if (both) {
                        const float4 y = *reinterpret_cast<const float4*>(theirs + c * (128 * 36) + lane * 36 + k);
                        x = make_float4(fmaf(y.x, g, x.x), fmaf(y.y, g, x.y), fmaf(y.z, g, x.z), fmaf(y.w, g, x.w));
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
                        const float4 y = *reinterpret_cast<const float4*>(stage + ro * 36 + e + 4);
                        if (row < tw.rows) {
                            const int t2 = row / p.group, h2 = h * p.group + row - t2 * p.group;
                            *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(q.q0 + t2) * p.out_stride +
                                                      static_cast<int64_t>(h2) * D + 32 * c + e) =
                                make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                                           pack_bf16(y.z, y.w));
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
        // softmax cuts K's columns, and V's get the scale byte 0 (a finite factor), as
        // P is 0 there; a bad page's tokens have block 0's, and the results are void.
        // Neighbouring groups of four lanes have neighbouring rows, whose
        // swizzles differ in the lowest bit: the stores meet no bank conflict.
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
        if (wg == kWgConvertK) {
            // unit k: row rr + 32 (k / NB), dims 64 (k % NB) + 16 (ct % 4) ..
            constexpr int NB = D / 64, KU = 4 * NB;
            const int rr = ct >> 2;
            const uint8_t* kbase = p.g.kcodes + (rr & 15) * D + 16 * (ct & 3);
            const uint8_t* sbase = p.g.kscale + (rr & 15);
            uint4 kr[KU];
            uint32_t ks[4];
            // rows rr + 32 m of tile j, whose block is `blk` of lane (rr >> 4) + 2 m
            auto fetch = [&](int m, uint32_t blk) {
                const uint64_t at = __shfl_sync(0xffffffffu, blk, (rr >> 4) + 2 * m);
#pragma unroll
                for (int n = 0; n < NB; ++n) kr[m * NB + n] = ldg_nc_na_v4(kbase + at * (16 * D) + 64 * n);
                ks[m] = ldg_early(sbase + at * 16);
            };
            int ahead = entry_at(1);
            if (T > 0) {
                const uint32_t blk = block_of(0, entry_at(0));
#pragma unroll
                for (int m = 0; m < 4; ++m) fetch(m, blk);
            }
            for (int j = 0; j < T; ++j) {
                const int st = j & 1;
                const uint32_t blk = block_of(j + 1, ahead);  // (block 0 past the last tile: read, not used)
                ahead = entry_at(j + 2);
                if (ok) ok = warp_wait(&bars[T_K_EMPTY + st], ((j >> 1) & 1) ^ 1, ab, kDevTimeoutConvert);
                if (!ok) continue;
                uint8_t* dst = smem + Lay::kK + st * Lay::kTile;
                uint8_t* lo = dst + bktile_off(rr, 16 * (ct & 3));
                uint8_t* hi = dst + bktile_off(rr, 16 * (ct & 3) + 8);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t f1 = scale_factor(ks[m]);
                    const uint32_t f[8] = {f1, f1, f1, f1, f1, f1, f1, f1};
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int off = n * (kTileN * 128) + m * (32 * 128);
                        put16(lo + off, hi + off, kr[m * NB + n], f);
                    }
                    fetch(m, blk);  // the next tile's rows, into the registers just freed
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[T_K_FULL + st]);
            }
        } else {
            // tokens 16 c .. of the dims d0 + 16 k
            constexpr int VU = D / 16;
            const int c = (ct & 3) | ((ct >> 4) & 4), d0 = (ct >> 2) & 15;
            uint4 vr[VU];
            uint4 vs = make_uint4(0, 0, 0, 0);
            // block `at` of 16 tokens: page and head at >> pb, place 16 (at mod 2^pb)
            auto source = [&](uint32_t at) {
                return p.g.vcodes + ((static_cast<uint64_t>(at >> pb) * D + d0) << p.g.page_shift) + 16 * (at & ((1u << pb) - 1u));
            };
            const uint32_t step = 16u << p.g.page_shift;  // 16 dims
            auto fetch_vs = [&](uint32_t at) {
                vs = ldg_nc_na_v4(p.g.vscale + static_cast<uint64_t>(at) * 16);
            };
            int ahead = entry_at(1);
            if (T > 0) {
                const uint32_t at = __shfl_sync(0xffffffffu, block_of(0, entry_at(0)), c);
                const uint8_t* src = source(at);
#pragma unroll
                for (int k = 0; k < VU; ++k) vr[k] = ldg_nc_na_v4(src + k * step);
                fetch_vs(at);
            }
            for (int j = 0; j < T; ++j) {
                const int st = j & 1;
                const uint32_t at = __shfl_sync(0xffffffffu, block_of(j + 1, ahead), c);
                ahead = entry_at(j + 2);
                if (ok) ok = warp_wait(&bars[T_V_EMPTY + st], ((j >> 1) & 1) ^ 1, ab, kDevTimeoutConvert);
                if (!ok) continue;
                uint32_t f[8];
                const uint4 cut = cut16(vs, q.kv - (j0 + j * kTileN + 16 * c));
                const uint32_t nan[4] = {__vcmpgtu4(cut.x, 0x86868686u), __vcmpgtu4(cut.y, 0x86868686u),
                                         __vcmpgtu4(cut.z, 0x86868686u), __vcmpgtu4(cut.w, 0x86868686u)};
                const uint32_t w[4] = {cut.x & ~nan[0], cut.y & ~nan[1], cut.z & ~nan[2], cut.w & ~nan[3]};
                // A V row that is not a number (scale byte over 134) counts as 0 in
                // the product; the rows that see it are marked.  Slot j & 3: each
                // group has looked at tile j - 4 before it handed over P of tile
                // j - 2, whose product freed this buffer.
                if ((warp & 1) == 0) {  // (the warps with the tokens' first dims: four blocks of 16 each)
                    if (lane < 4) *reinterpret_cast<uint4*>(smem + Lay::kScale + (j & 3) * kTileN + 16 * c) = cut;
                    const bool bad = __any_sync(0xffffffffu, (nan[0] | nan[1] | nan[2] | nan[3]) != 0u);
                    if (lane == 0) misc[4 + 4 * ((warp >> 1) & 1) + (j & 3)] = bad ? 1u : 0u;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = factors02(w[k]);
                    f[2 * k + 1] = factors13(w[k]);
                }
                fetch_vs(at);
                const uint8_t* src = source(at);
                uint8_t* dst = smem + Lay::kV + st * Lay::kTile;
                uint8_t* lo = dst + bvtile_off(d0, 16 * c, D);
                uint8_t* hi = dst + bvtile_off(d0, 16 * c + 8, D);
#pragma unroll
                for (int k = 0; k < VU; ++k) {
                    put16(lo + 16 * 128 * k, hi + 16 * 128 * k, vr[k], f);
                    vr[k] = ldg_nc_na_v4(src + k * step);  // the next tile's, into the registers just freed
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[T_V_FULL + st]);
            }
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
    static std::atomic<uint64_t> configured{0};
    constexpr uint32_t smem = TcLayout<D>::kAlloc;
    static_assert(smem <= 227 * 1024, "shared memory over the sm_103 limit");
    const TilesKernel kernel{paged_tc_kernel<D>, configured};
    return launch_tiles<D>(kernel, kernel, smem, p, part_floats_max, s);  // (few is 0: never by number)
}

}  // namespace

cudaError_t launch_paged_tc(PagedAttnParams& p, int D, size_t part_floats_max, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, part_floats_max, s) : launch_d<64>(p, part_floats_max, s);
}

}  // namespace rc
