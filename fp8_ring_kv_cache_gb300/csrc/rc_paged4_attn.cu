// rc_paged4_attn.cu -- attention of few query rows over the 4-bit pages.
//
// The rows of a KV head (its sequence's new tokens x the query heads that share it)
// are 32 at most, in tiles of 8 or 16.  Bound by reading the codes, and as much by
// turning them into numbers.  The work is a line of units, a unit being 256 cached
// tokens of a (sequence, KV head): each block has an equal stretch of that line, whatever the sequences'
// lengths are, and finds its place by a sum over the lengths.  (Where all there can be
// is little, a block's place is its place in the grid: the sum takes 1.5 us.)  A list
// that a block has only a part of leaves its (maximum, sum, O) in the workspace, and the
// last of the blocks that share it joins them in the blocks' order, so that results do
// not depend on timing.
// A warp takes 64 cached tokens of a unit at a time, transposed, so that the few rows
// are the short side of the products (m16n8k16, fp16 operands, fp32 sums):
//   S^T = K Q^T      a lane's 16 bytes of a K row are 32 of the summed dims for its
//                    token; which dims of a product they are is free as long as Q is
//                    held in the same order.  Rows of Q are scaled to fp16's range.
//   P = exp2(S - max + 14), online, rounded to fp16 (2^-12 of each weight; weights down
//                    to 2^-28 of the largest keep all their bits, the row sums are
//                    not rounded; scores from 2^20 on: kLargeScore4); an 8 x 8 transpose of the accumulators makes them
//                    the B operand of
//   O^T += V^T P^T   whose A operand is an 8-byte piece of a V row: 16 tokens of one dim.
//                    The tokens of S's rows are chosen to match.
// One conversion makes two codes exact fp16 numbers and one multiplication scales
// them, exactly: a code times a scale has 6 bits.  A scale byte is an fp16 number but
// for a shift.
// A warp's codes and scales go through shared memory of its own, by asynchronous copies:
// the next K tokens are on their way from when this chunk's scores are done, the next V
// from when its products are.  V's scales are made fp16 once a chunk by one lane each,
// and read by all.
// 32 single tokens (sequences of 61 to 16,381 tokens, 8 KV heads x 6 query heads x 128):
// 62.5 us for 304 MB, 0.73 of the rate of a copy.  The copies alone take 55 us, the
// arithmetic alone 54: neither hides the other wholly.  (Codes straight into registers, a
// block a fixed split: 76 us.  Looking for large scores is in the 62.5 with 0.6 us; the
// times at the rules below were taken without it.)
#include <algorithm>
#include <type_traits>

#include "rc_paged4.cuh"

namespace rc {

namespace {

constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kChunk = 64;                  // cached tokens of a warp's step
constexpr int kUnit = kRowsWarps * kChunk;  // cached tokens of a unit of work
constexpr float kWeightShift = 14.f;        // log2 of the largest weight in fp16

// A part's result in the workspace: O [rows][D], then max and sum [rows] each.
template <int D, int NR>
constexpr int part_floats() {
    return 8 * NR * D + 2 * 8 * NR;
}

// Weight of a partial whose running max is m against the joint max M (both in
// log2 units; -inf: the partial saw nothing).
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }

// Sequence s, without new tokens if it has more rows than this kernel takes.
__device__ __forceinline__ Seq rows_seq(const PagedAttnParams& p, int s) {
    Seq q = load_seq(p.g, s);
    if (q.n * p.group > p.most) q.n = 0;
    return q;
}

// Units of a sequence, for one KV head: none without new tokens, one at least with some.
__device__ __forceinline__ int units_of(const Seq& q) { return q.n == 0 ? 0 : max(1, (q.kv + kUnit - 1) / kUnit); }

// A warp's 64 cached tokens in shared memory, as blocks of 16: K's codes [16][D / 2] and scales [D / 16][16] a block, V's
// codes [D][4 blocks][8 bytes] and scales [D / 16][4 blocks][16], and these as fp16.  (D = 64: K's blocks lie 64 bytes
// apart, so that the lanes' reads meet no bank conflict.)
template <int D>
struct Stage {
    static constexpr int NB = D / 16;
    static constexpr int kKBlock = 16 * D / 2 + (D == 64 ? 64 : 0);
    static constexpr int kK = 0;
    static constexpr int kKScale = kK + 4 * kKBlock;
    static constexpr int kV = kKScale + 64 * NB;
    static constexpr int kVScale = kV + 32 * D;
    static constexpr int kVFactor = kVScale + 64 * NB;
    static constexpr int kBytes = kVFactor + 128 * NB;
};

// A block's shared memory.
template <int D, int NR>
struct RowsSmem {
    static constexpr int kRowTile = 8 * NR, kRow = D + 4;  // O's rows lie where a warp's tokens were
    static constexpr int kApart = Stage<D>::kBytes > kRowTile * kRow * 4 ? Stage<D>::kBytes : kRowTile * kRow * 4;
    uint8_t stages[kRowsWarps][kApart];
    float m[kRowsWarps][kRowTile], l[kRowsWarps][kRowTile];
    int last;
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a block does at a time: units k0 .. k1 - 1 of a list.  A list is a KV head of sequence s, or one of its row tiles:
// number h = head x row tiles + tile.
struct Piece {
    Seq q;
    int s, h, k0, k1;
    bool whole;  // the list has no others
    // else: the place of this part's result in the workspace, that of the list's first one, how many there are, how far
    // apart they lie (the first is one place nearer to the second if `odd`), and their counter
    int mine, first, parts, step, odd, counter;
};

// Blocks of an SM: registers spilled cost more than fewer warps (one sequence of 131,072 tokens x 8 heads x 128 with a
// row: 4 blocks of 128 registers 46 us, 3 of 162 41; 32 x 8,000 with 16 rows: 3 blocks 90 us, 2 81).
constexpr int grid_blocks(int NR) { return NR == 1 ? 4 : 2; }
constexpr int line_blocks(int NR) { return NR == 1 ? 3 : 2; }

// 8 NR rows (NR 1 or 2).
template <int D, int NR>
__device__ __forceinline__ void attend_piece(const PagedAttnParams& p, RowsSmem<D, NR>& sh, const Piece& pc) {
    using St = Stage<D>;
    using Sh = RowsSmem<D, NR>;
    constexpr int KW = D / 32;  // words of a K row that a lane reads
    constexpr int KB = D / 64;  // blocks of 16 dims among them
    constexpr int MT = D / 16;  // m tiles of O^T: blocks of 16 dims
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const Seq& q = pc.q;
    const int s = pc.s, h = pc.h / p.row_tiles, row0 = (pc.h - h * p.row_tiles) * (8 * NR);
    const int rows = min(8 * NR, q.n * p.group - row0);
    if (rows <= 0) return;  // (so do the list's other parts)
    const int j0 = pc.k0 * kUnit, j1 = min(q.kv, pc.k1 * kUnit);
    uint8_t* st = sh.stages[warp];
    const int P = 1 << p.g.page_shift;

    // ---- the copies of a chunk of 64 tokens.  Lane l's page is that of the chunk's block l % 4, looked up a chunk ahead.  A
    // block behind the sequence's end, or on a bad page, is read from page 0 instead.  Tokens behind the end are cut off (K)
    // and given the scale 0 (V); those on a bad page have page 0's scores and the scale 0: that call's results are void.
    const uint32_t* pages =
        reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
    auto entry = [&](int jc) {
        const int j = jc + 16 * t;
        return jc < j1 && j < q.kv ? static_cast<int>(ldg_early(pages + (j >> p.g.page_shift))) : 0;
    };
    // page x kv_heads + head of the lane's block; ok: there is such a block
    auto block_at = [&](int jc, int page, bool& ok) {
        ok = jc < j1 && jc + 16 * t < q.kv && check_page(p.g, page);
        return (ok ? static_cast<uint32_t>(page) : 0u) * p.g.kv_heads + h;
    };
    // (at: page x kv_heads + head; a page's blocks of a chunk lie where they lie in every chunk, or for pages of 128 tokens
    // in its other half)
    const int half = P == 128 ? kChunk : 0;
    auto fetch_k = [&](int jc, uint32_t at) {
        {
            const int b = lane >> 3;
            const uint32_t page = __shfl_sync(0xffffffffu, at, b), off = (16 * b & (P - 1)) + (jc & half);
            const uint8_t* src = p.g.kcodes + 16 * (lane & 7) + off * (D / 2) + static_cast<uint64_t>(page) * static_cast<uint32_t>(P * (D / 2));
            uint8_t* dst = st + St::kK + b * St::kKBlock + 16 * (lane & 7);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) cp_async16(dst + 128 * j, src + 128 * j);
        }
        {
            const int b = lane / MT & 3, nb = lane & (MT - 1);
            const uint32_t page = __shfl_sync(0xffffffffu, at, b), off = (16 * b & (P - 1)) + (jc & half);
            if (D == 128 || lane < 4 * MT)
                cp_async16(st + St::kKScale + 16 * lane, p.g.kscale + nb * P + off + static_cast<uint64_t>(page) * static_cast<uint32_t>(P * MT));
        }
    };
    auto fetch_v = [&](int jc, uint32_t at) {
        if (P >= 32) {  // two blocks lie side by side
            const int b = 2 * (lane & 1), d = lane >> 1;
            const uint32_t page = __shfl_sync(0xffffffffu, at, b), off = (16 * b & (P - 1)) + (jc & half);
            const uint8_t* src = p.g.vcodes + (d * P + off) / 2 + static_cast<uint64_t>(page) * static_cast<uint32_t>(P * (D / 2));
            uint8_t* dst = st + St::kV + 32 * d + 8 * b;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) cp_async16(dst + 512 * j, src + 8 * P * j);
        } else {
            const int b = lane & 3, d = lane >> 2;
            const uint8_t* src = p.g.vcodes + 8 * d + static_cast<uint64_t>(at) * (8 * D);
            uint8_t* dst = st + St::kV + 32 * d + 8 * b;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) cp_async8(dst + 256 * j, src + 64 * j);
        }
        const int nb = lane >> 2;
        if (D == 128 || nb < MT)
            cp_async16(st + St::kVScale + 16 * lane,
                       p.g.vscale + nb * P + (16 * t & (P - 1)) + (jc & half) + static_cast<uint64_t>(at) * static_cast<uint32_t>(P * MT));
    };
    constexpr int kStride = kRowsWarps * kChunk;
    int jc = j0 + warp * kChunk;
    int ahead = entry(jc);
    int after = entry(jc + kStride);

    // ---- the query rows, on their way with the first page
    const __nv_bfloat16* qrow[NR];
    bool live[NR];
    // of the rows 2 t + x of each eight, whose scores the lane gets: tokens seen
    // (rows past the end see all; nothing of theirs is stored)
    int limit[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int rr = row0 + 8 * r + g;
        live[r] = rr < row0 + rows;
        const int tok = live[r] ? rr / p.group : 0, head = h * p.group + (live[r] ? rr - tok * p.group : 0);
        qrow[r] = p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D;
        const int lim = !live[r] ? 1 << 30 : p.causal ? max(0, q.kv - q.n + tok + 1) : q.kv;
#pragma unroll
        for (int x = 0; x < 2; ++x) limit[r][x] = __shfl_sync(0xffffffffu, lim, 4 * (2 * t + x));
    }
    uint32_t qb[NR][D / 16][2];
    float qscale[NR][2];
    bool vok;  // the lane's block of the chunk whose V is on its way
    {
        const uint32_t at = block_at(jc, ahead, vok);
        ahead = after;
        if (jc < j1) fetch_k(jc, at);
        cp_async_commit();
        if (jc < j1) fetch_v(jc, at);
        cp_async_commit();
    }
    query_tile_f16<D, NR, D / 4>(qrow, live, p.sm_log2, qb, qscale);
    bool may_be_large = false;  // (rows of zeros are taken for such, but for those past the end)
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) may_be_large |= limit[r][x] != 1 << 30 && qscale[r][x] >= p.sm_log2 * kLargeQuery4;
    may_be_large = __any_sync(0xffffffffu, may_be_large);
    // what every row sees
    const int least = min(j1, p.causal ? max(0, q.kv - q.n + 1) : q.kv);

    float o[NR][MT][4];
    float m_run[NR][2], l_run[NR][2];  // m_run: 14 below the maximum
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[r][n][i] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            m_run[r][x] = -INFINITY;
            l_run[r][x] = 0.f;
        }
    }
    for (; jc < j1; jc += kStride) {
        const bool more = jc + kStride < j1;
        const int kblk = jc + 16 * (g >> 1);
        bool next_ok;
        const uint32_t next = block_at(jc + kStride, ahead, next_ok);
        ahead = entry(jc + 2 * kStride);
        cp_async_wait<1>();  // K is there
        __syncwarp();
        // m tile i of S^T: its row g is token kblk + 4 i + (g & 1), its row g + 8 the next but one
        float sc[NR][4][4];
        {
            const uint8_t* kp = st + St::kK + (g >> 1) * St::kKBlock + (g & 1) * (D / 2) + t * (D / 8);
            uint4 ksw[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b)
                ksw[b] = *reinterpret_cast<const uint4*>(st + St::kKScale + (g >> 1) * (16 * MT) + (KB * t + b) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[r][i][k] = 0.f;
                uint32_t f[KB], kw[2][KW];  // f: the scales of the tile's two tokens
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const uint32_t w = i == 0 ? ksw[b].x : i == 1 ? ksw[b].y : i == 2 ? ksw[b].z : ksw[b].w;
                    f[b] = scales_apart(w, g & 1);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint8_t* from = kp + (4 * i + 2 * x) * (D / 2);
                    if constexpr (KW == 4) {
                        const uint4 w = *reinterpret_cast<const uint4*>(from);
                        kw[x][0] = w.x, kw[x][1] = w.y, kw[x][2] = w.z, kw[x][3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(from);
                        kw[x][0] = w.x, kw[x][1] = w.y;
                    }
                }
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    uint32_t wa[4], wb[4];
                    codes8_f16(kw[0][k], wa);
                    codes8_f16(kw[1][k], wb);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t a[4] = {half2_mul_lo(wa[2 * c], f[k / 2]), half2_mul_hi(wb[2 * c], f[k / 2]),
                                               half2_mul_lo(wa[2 * c + 1], f[k / 2]), half2_mul_hi(wb[2 * c + 1], f[k / 2])};
#pragma unroll
                        for (int r = 0; r < NR; ++r) mma_f16(sc[r][i], a, qb[r][2 * k + c][0], qb[r][2 * k + c][1]);
                    }
                }
            }
        }
        __syncwarp();
        if (more) fetch_k(jc + kStride, next);  // the next chunk's, where this one's has been read
        cp_async_commit();

        // softmax: scores 2 a + x of m tile i: token kblk + 4 i + 2 a + (g & 1), row 2 t + x
        const bool full = jc + kChunk <= least;
        if (!full) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int j = kblk + 4 * i + 2 * a + (g & 1);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (j >= limit[r][x] || j >= j1) sc[r][i][2 * a + x] = -INFINITY;
                }
        }
        bool moved = false;
        float alpha[NR][2];
        auto softmax = [&](auto large) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = max3(mx, sc[r][i][x], sc[r][i][2 + x]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    float m_new = fmaxf(m_run[r][x], fmaf(mx, qscale[r][x], -kWeightShift));
                    const bool far = large && m_new != -INFINITY && fabsf(m_new) >= kLargeScore4;
                    if (far) m_new = fmaxf(m_run[r][x], __fmul_rn(mx, qscale[r][x]));
                    const float base = m_new == -INFINITY ? 0.f : m_new;
                    alpha[r][x] = ex2(m_run[r][x] - base);  // 0 while nothing was seen
                    m_run[r][x] = m_new;
                    moved |= alpha[r][x] != 1.f;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            const float v = sc[r][i][2 * a + x];
                            const float w = ex2(far ? __fadd_rn(__fmul_rn(v, qscale[r][x]), -base) : fmaf(v, qscale[r][x], -base));
                            sc[r][i][2 * a + x] = w;
                            sum += w;
                        }
                    l_run[r][x] = l_run[r][x] * alpha[r][x] + sum;
                }
        };
        if (may_be_large)
            softmax(std::true_type{});
        else
            softmax(std::false_type{});
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int n = 0; n < MT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][n][i] *= alpha[r][i & 1];
        }
        cp_async_wait<1>();  // V is there
        __syncwarp();
        // V's scales as fp16, once for the warp: a lane has those of block lane / 4 of the dims for block t of the tokens
        if (D == 128 || lane < 4 * MT) {
            const uint4 w = *reinterpret_cast<const uint4*>(st + St::kVScale + 16 * lane);
            uint32_t vs[4] = {w.x, w.y, w.z, w.w}, nans = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) nans |= nan_scales(vs[i]);
            if (!full || nans != 0 || !vok) {
                // scale 0 for tokens that the sequence does not have, or whose V is not a number
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int left = vok ? q.kv - (jc + 16 * t + 4 * i) : 0;  // tokens of the word that exist
                    const uint32_t have = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                    vs[i] &= have & ~__vcmpgtu4(vs[i], 0x01010101u * (kFirstNan4 - 1));
                }
            }
            uint4* to = reinterpret_cast<uint4*>(st + St::kVFactor + 32 * lane);
            to[0] = make_uint4(scales01(vs[0]), scales23(vs[0]), scales01(vs[1]), scales23(vs[1]));
            to[1] = make_uint4(scales01(vs[2]), scales23(vs[2]), scales01(vs[3]), scales23(vs[3]));
            vok = vok && nans == 0;
        }
        if (__any_sync(0xffffffffu, !vok)) {
            // A token whose V is not a number (its first block says so) must reach the rows that see it and no other, so
            // that is moved from V (0 x NaN would reach every row) into the weights.
            const uint4 w = *reinterpret_cast<const uint4*>(st + St::kVScale + 16 * (g >> 1));
            const uint32_t theirs[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int j = kblk + 4 * i + 2 * a + (g & 1);
                    if (((theirs[i] >> (8 * (2 * a + (g & 1)))) & 0xffu) >= kFirstNan4) {
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (j < limit[r][x] && j < j1) sc[r][i][2 * a + x] = __uint_as_float(0x7fc00000u);
                    }
                }
        }
        uint32_t pb[NR][4][2];  // products over tokens 16 t + 4 i + 2 a + {0, 1} of the chunk
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int a = 0; a < 2; ++a) pb[r][i][a] = transpose8(pack_f16(sc[r][i][2 * a], sc[r][i][2 * a + 1]));
        __syncwarp();
        const uint8_t* vp = st + St::kV + 32 * g + 8 * t;
#pragma unroll
        for (int n = 0; n < MT; ++n) {
            const uint2 v0 = *reinterpret_cast<const uint2*>(vp + 512 * n), v1 = *reinterpret_cast<const uint2*>(vp + 512 * n + 256);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint4 f = *reinterpret_cast<const uint4*>(st + St::kVFactor + 128 * n + 32 * t + 16 * w);
                uint32_t lo[4], hi[4];
                codes8_f16(w ? v0.y : v0.x, lo);
                codes8_f16(w ? v1.y : v1.x, hi);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t f0 = c ? f.z : f.x, f1 = c ? f.w : f.y;
                    const uint32_t a[4] = {half2_mul(lo[2 * c], f0), half2_mul(hi[2 * c], f0), half2_mul(lo[2 * c + 1], f1),
                                           half2_mul(hi[2 * c + 1], f1)};
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(o[r][n], a, pb[r][2 * w + c][0], pb[r][2 * w + c][1]);
                }
            }
        }
        __syncwarp();
        if (more) fetch_v(jc + kStride, next);
        cp_async_commit();
        vok = next_ok;
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the warps: each leaves its O where its chunks were
    float* so = reinterpret_cast<float*>(&sh.stages[0][0]);
    constexpr int kRowTile = Sh::kRowTile, kStage = Sh::kApart / 4, kRow = Sh::kRow;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float l = l_run[r][x];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int row = 8 * r + 2 * t + x;
            if (g == 0) {
                sh.m[warp][row] = m_run[r][x];
                sh.l[warp][row] = l;
            }
#pragma unroll
            for (int n = 0; n < MT; ++n) {
                so[warp * kStage + row * kRow + 16 * n + g] = o[r][n][x];
                so[warp * kStage + row * kRow + 16 * n + 8 + g] = o[r][n][2 + x];
            }
        }
    __syncthreads();
    auto store_out = [&](int r, int d, float4 v, float M, float L) {
        const int tok = (row0 + r) / p.group, head = h * p.group + row0 + r - tok * p.group;
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // a sum that is not a number stays one
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(q.q0 + tok) * p.out_stride +
                                  static_cast<int64_t>(head) * D + d) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        if (d == 0 && p.lse != nullptr)
            p.lse[static_cast<int64_t>(q.q0 + tok) * p.heads + head] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    constexpr int kPart = part_floats<D, NR>();
    float* const mine = p.part + static_cast<size_t>(pc.mine) * kPart;
    for (int i = tid; i < rows * (D / 4); i += kRowsThreads) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sh.m[w][r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) {
            const float f = join_weight(sh.m[w][r], M);
            const float4 v = *reinterpret_cast<const float4*>(so + w * kStage + r * kRow + d);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
            L += f * sh.l[w][r];
        }
        if (pc.whole) {
            store_out(r, d, acc, M, L);
        } else {
            *reinterpret_cast<float4*>(mine + r * D + d) = acc;
            if (d == 0) {
                mine[kRowTile * D + r] = M;
                mine[kRowTile * D + kRowTile + r] = L;
            }
        }
    }
    if (pc.whole) return;
    // ---- join the parts, in the block of the last one to arrive
    const int parts = pc.parts;
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        int* const counter = p.counters + pc.counter;
        const bool is = atomicAdd(counter, 1) == parts - 1;
        if (is) *counter = 0;
        __threadfence();
        sh.last = is;
    }
    __syncthreads();
    if (!sh.last) return;
    auto part = [&](int i) { return p.part + static_cast<size_t>(pc.first + (i == 0 ? 0 : i * pc.step - pc.odd)) * kPart; };
    // a row's maximum and sum by some lanes of one warp
    constexpr int kLanes = kRowsThreads / kRowTile;  // 8 or 16
    const int row = tid / kLanes;
    float M = -INFINITY, L = 0.f;
    if (row < rows)
        for (int i = tid % kLanes; i < parts; i += kLanes) {
            const float* b = part(i) + kRowTile * D + row;
            const float m = __ldcg(b), l = __ldcg(b + kRowTile), top = fmaxf(M, m);
            L = L * join_weight(M, top) + l * join_weight(m, top);
            M = top;
        }
    float top = M;
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    L *= join_weight(M, top);
#pragma unroll
    for (int x = kLanes / 2; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
    if (tid % kLanes == 0) {
        sh.m[0][row] = top;
        sh.l[0][row] = L;
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kRowsThreads) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 16;  // loads on the way
        for (int k = 0; k < parts; k += kBatch) {
            float4 v[kBatch];
            float m[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const float* b = part(min(k + x, parts - 1));
                v[x] = __ldcg(reinterpret_cast<const float4*>(b + r * D + d));
                m[x] = __ldcg(b + kRowTile * D + r);
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const float w = k + x < parts ? join_weight(m[x], sh.m[0][r]) : 0.f;
                acc.x += w * v[x].x;
                acc.y += w * v[x].y;
                acc.z += w * v[x].z;
                acc.w += w * v[x].w;
            }
        }
        store_out(r, d, acc, sh.m[0][r], sh.l[0][r]);
    }
}

// ---------------------------------------------------------------- a block's place in the grid
template <int D, int NR>
__global__ void __launch_bounds__(kRowsThreads, grid_blocks(NR)) paged4_rows_kernel(PagedAttnParams p) {
    __shared__ __align__(16) RowsSmem<D, NR> sh;
    Piece pc;
    pc.s = blockIdx.z;
    pc.h = blockIdx.y;
    pc.q = rows_seq(p, pc.s);
    const int units = units_of(pc.q), per = p.split_tokens / kUnit;
    pc.k0 = blockIdx.x * per;
    if (pc.k0 >= units) return;
    pc.k1 = min(units, pc.k0 + per);
    pc.parts = (units + per - 1) / per;
    pc.whole = pc.parts == 1;
    pc.counter = pc.s * gridDim.y + pc.h;
    pc.first = pc.counter * p.splits;
    pc.mine = pc.first + blockIdx.x;
    pc.step = 1;
    pc.odd = 0;
    attend_piece<D, NR>(p, sh, pc);
}

// ---------------------------------------------------------------- a block's stretch of the line
// a / b >= 0, in 32 bits where they do.
__device__ __forceinline__ int64_t divide_line(int64_t a, int64_t b) {
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A list is `gap` units longer on the line than it is, which stand for its start and end (32 sequences of 61 to 16,381
// tokens x 8 heads x 128: 72 us without, 67 with).
struct Line {
    int64_t units;
    int blocks, gap;

    __device__ __forceinline__ int64_t cut(int block) const { return divide_line(units * block, blocks); }  // its first unit
    __device__ __forceinline__ int block_of(int64_t unit) const {
        return static_cast<int>(divide_line((unit + 1) * blocks - 1, units));
    }
};

template <int D, int NR>
__global__ void __launch_bounds__(kRowsThreads, line_blocks(NR)) paged4_line_kernel(PagedAttnParams p) {
    __shared__ __align__(16) RowsSmem<D, NR> sh;
    __shared__ Line line;
    __shared__ int64_t u_end;
    __shared__ int sums[2][kRowsWarps];
    __shared__ Piece start;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, hk = p.g.kv_heads * p.row_tiles;  // lists of a sequence

    // ---- a thread sums over `per` sequences (512 at most, of 65,536 units at most)
    const int per = (p.g.seqs + kRowsThreads - 1) / kRowsThreads;
    const int s_first = min(p.g.seqs, tid * per), s_end = min(p.g.seqs, s_first + per);
    int units = 0, lists = 0;
    for (int s = s_first; s < s_end; ++s) {
        const int n = units_of(rows_seq(p, s));
        units += n;
        lists += n > 0;
    }
    int u_to = units, l_to = lists;  // up to and with the thread's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, u_to, o), y = __shfl_up_sync(0xffffffffu, l_to, o);
        if (lane >= o) {
            u_to += x;
            l_to += y;
        }
    }
    if (lane == 31) {
        sums[0][warp] = u_to;
        sums[1][warp] = l_to;
    }
    __syncthreads();
    int64_t u_all = 0, l_all = 0, before = u_to - units, l_before = l_to - lists;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
        if (w < warp) {
            before += sums[0][w];
            l_before += sums[1][w];
        }
        u_all += sums[0][w];
        l_all += sums[1][w];
    }
    if (u_all == 0) return;
    u_all *= hk;
    l_all *= hk;
    int64_t u;
    {
        // two units a block at least
        Line l;
        l.blocks = static_cast<int>(max(static_cast<int64_t>(1), min(u_all / 2, static_cast<int64_t>(gridDim.x))));
        l.gap = u_all >= 4 * static_cast<int64_t>(l.blocks) ? 1 : 0;
        l.units = u_all + l.gap * l_all;
        if (blockIdx.x >= l.blocks) return;
        u = l.cut(blockIdx.x);
        before = (before + l.gap * l_before) * hk;
        if (tid == 0) {
            line = l;
            u_end = l.cut(blockIdx.x + 1);
        }
        if (before <= u && u < before + (units + static_cast<int64_t>(l.gap) * lists) * hk) {  // one thread: the place of u
            for (int s = s_first; s < s_end; ++s) {
                const Seq q = rows_seq(p, s);
                const int n = units_of(q) + l.gap;
                const int64_t all = q.n == 0 ? 0 : static_cast<int64_t>(n) * hk;
                if (u < before + all) {
                    start.q = q;
                    start.s = s;
                    start.h = static_cast<int>(divide_line(u - before, n));
                    start.k0 = static_cast<int>(u - before - static_cast<int64_t>(start.h) * n);
                    break;
                }
                before += all;
            }
        }
    }
    __syncthreads();
    Piece pc;
    pc.q = start.q;
    pc.s = start.s;
    pc.h = start.h;
    pc.k0 = start.k0;
    while (true) {
        const int list = units_of(pc.q);
        const int stretch = static_cast<int>(min(static_cast<int64_t>(list + line.gap - pc.k0), u_end - u));
        if (pc.k0 < list) {
            pc.k1 = min(list, pc.k0 + stretch);
            pc.whole = pc.k0 == 0 && pc.k1 == list;
            if (!pc.whole) {
                // The block with a list's beginning has its result in its second place in the workspace, the others, whose
                // stretches begin inside it, in their first.
                const int b0 = line.block_of(u - pc.k0);
                pc.parts = line.block_of(u - pc.k0 + list - 1) - b0 + 1;
                pc.counter = b0;
                pc.first = 2 * b0 + 1;
                pc.mine = 2 * static_cast<int>(blockIdx.x) + (pc.k0 == 0 ? 1 : 0);
                pc.step = 2;
                pc.odd = 1;
            }
            attend_piece<D, NR>(p, sh, pc);
        }
        u += stretch;
        if (u >= u_end) break;
        pc.k0 = 0;
        if (++pc.h == hk) {
            pc.h = 0;
            do {  // (u is in the line: there is one)
                pc.q = rows_seq(p, ++pc.s);
            } while (pc.q.n == 0 && pc.s + 1 < p.g.seqs);
        }
        __syncthreads();
    }
}

// Of the sequences with `rows` rows a KV head at most.
template <int D, int NR>
cudaError_t launch_rows(PagedAttnParams& p, int64_t rows, cudaStream_t s) {
    constexpr int kGrid = 152 * grid_blocks(NR), kLine = 152 * line_blocks(NR);  // blocks at once
    constexpr int kPlaces = kGrid > 2 * kLine ? kGrid : 2 * kLine;
    static_assert(kPlaces * part_floats<D, NR>() * sizeof(float) <= (32u << 20) && kPlaces <= 16384, "places in the workspace");
    // The grid's way while all blocks are there at once with four units each at most: 64 sequences x 1,000 tokens x 8 heads
    // 19.9 us, 25.6 as a line; 8 x 2,000 12.4 and 15.2; one of 4,000 8.4 and 11.5; one of 337 x 2 heads x 64 5.3 and 6.6.
    // (Two units stay together, but for few blocks.)
    p.most = static_cast<int>(rows);
    p.row_tiles = static_cast<int>((rows + 8 * NR - 1) / (8 * NR));
    const int64_t lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads * p.row_tiles;
    const int64_t units = std::max(1, (p.g.max_kv + kUnit - 1) / kUnit);
    int64_t splits = std::min<int64_t>(std::max<int64_t>(kGrid / lists, 1), units);
    const int64_t least = units > 2 && lists * splits <= 2 * 152 ? 1 : 2;
    const int64_t per = std::max((units + splits - 1) / splits, least);
    splits = (units + per - 1) / per;
    if (lists * splits <= kGrid && per <= 4) {
        p.split_tokens = static_cast<int>(per) * kUnit;
        p.splits = static_cast<int>(splits);
        paged4_rows_kernel<D, NR><<<dim3(p.splits, p.g.kv_heads * p.row_tiles, p.g.seqs), kRowsThreads, 0, s>>>(p);
    } else {
        paged4_line_kernel<D, NR><<<kLine, kRowsThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

// Up to 32 rows per KV head as tiles of 8 or 16 rows, which read the codes again (the second time from L2, mostly): 32
// sequences x 8,000 tokens x 8 KV heads x 128 with 32 rows 146 us, 199 as a tile of the tcgen05 kernel, which takes as
// long for 17 rows as for 128; 9 of 1,021 to 12,007 with 20 rows 47 and 78; 16 of 500 with 32 rows 10.4 and 15.3.  With 48
// rows 210 us against 200.
constexpr int kRowsFew = 32;

template <int D>
cudaError_t launch_attention_d(PagedAttnParams& p, size_t part_floats_max, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    if (rows <= 8) return launch_rows<D, 1>(p, rows, s);
    if (rows <= kRowsFew) return launch_rows<D, 2>(p, rows, s);
    // With long sequences in the call, those of a token or a few (what fills the row tiles that one token needs) have a
    // launch of their own, if as many as half of the sequences can be such.  All with 8,000 cached, 8 x 6 heads x 128: 63 single
    // tokens and a chunk of 512 take 222 us so, 472 in one kernel (as two calls 217); 31 and a chunk of 128 176 and 217 (as
    // two calls 94: the chunk alone is split); one and a chunk of 512 123 and 111, as the chunk leaves SMs free; 7 of 40
    // tokens and one of 300, where none is short, 69 and 70.
    if (p.group <= kRowsFew) {
        const int one = p.group <= 8 ? 8 : (p.group + 15) / 16 * 16, few = one / p.group;
        if (p.g.seqs > 1 && 2 * static_cast<int64_t>(p.g.tokens) <= static_cast<int64_t>(p.g.seqs) * (p.g.max_new + few)) {
            const cudaError_t e = one == 8 ? launch_rows<D, 1>(p, one, s) : launch_rows<D, 2>(p, one, s);
            if (e != cudaSuccess) return e;
            p.few = one;
        }
    }
    return launch_paged4_tc(p, D, part_floats_max, s);
}

}  // namespace

cudaError_t launch_paged4_attention(PagedAttnParams& p, int D, size_t part_floats_max, cudaStream_t s) {
    return D == 128 ? launch_attention_d<128>(p, part_floats_max, s) : launch_attention_d<64>(p, part_floats_max, s);
}

}  // namespace rc
