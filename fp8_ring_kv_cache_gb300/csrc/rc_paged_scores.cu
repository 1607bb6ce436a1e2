// rc_paged_scores.cu -- the attention weight that each cached token received:
// out[j] = scores[j] + sum over the query rows of exp(q . k_j scale - lse).
//
// paged_scores_few_kernel, for one tile of query rows (a decode step): bound by
// reading the K codes.  The rows stay in registers while the warps go over the
// cached tokens 64 at a time, reading K pieces straight into the fp16 products'
// operands as the attention does; the four lanes that hold a token's rows add up
// by halves, so that each ends with the sums of two tokens.  16 sequences of 509
// to 8,191 tokens x 8 KV heads x 6 query heads x 128: 17.6 us (76 MB, 11.3 us at the
// rate of a copy); the start of each block, three loads after one another, is what
// keeps it from there.
//
// paged_scores_rows_kernel, for some tiles of rows.
// A warp owns 32 cached tokens of one (sequence, KV head), decodes their K rows
// to bf16 once, into the registers where the matrix instructions want them, and
// goes over the head's query rows 16 at a time.  A token's sum stays with its
// owner, so no two threads add to one entry and the order is fixed.
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kScoreWarps = 4;
constexpr int kScoreTokens = 32;  // of a warp
constexpr int kScoreRowsMax = 32;  // of the kernels here

constexpr int kFewChunk = 64;  // cached tokens of a warp's step

// 8 NR rows; a block has `range` cached tokens (a multiple of 256).  Blocks an SM
// (8 KV heads x 128, 32 sequences of 8,000 tokens): 8 rows, as many as 78
// registers allow 59.6 us, 7 45.0, 8 48.4; 16 rows 4 54.5 us, 5 55.8, 6 62.4 (and
// with head_dim 64 33.8, 32.1, 36.3).
template <int D, int NR>
__global__ void __launch_bounds__(kScoreWarps * 32, NR == 1 ? 7 : D == 64 ? 5 : 4) paged_scores_few_kernel(PagedScoreParams p, int range) {
    constexpr int CH = D / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, s = blockIdx.z;
    const int j0 = blockIdx.x * range, stop = min(p.g.max_kv, j0 + range);
    const Seq q = load_seq(p.g, s);
    const int rows = q.n * p.group;
    const int64_t at = (static_cast<int64_t>(s) * p.g.kv_heads + h) * p.score_stride;
    const int end = rows > 0 ? min(stop, q.kv) : j0;  // tokens from here on keep their scores
    constexpr int kStride = kScoreWarps * kFewChunk;
    uint32_t qb[NR][D / 16][2];
    float qscale[NR][2], minus[NR][2];  // of rows 2 t + x, whose scores the lane gets
    int limit[NR][2];
    if (j0 < end) {
        const __nv_bfloat16* qrow[NR];
        bool live[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int rr = 8 * r + g;
            live[r] = rr < rows;
            const int tok = live[r] ? rr / p.group : 0, head = h * p.group + (live[r] ? rr - tok * p.group : 0);
            qrow[r] = p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D;
            const float lse = live[r] ? __ldg(p.lse + static_cast<int64_t>(q.q0 + tok) * p.heads + head) : -INFINITY;
            const int lim = lse == -INFINITY ? 0 : p.causal ? q.kv - q.n + tok + 1 : q.kv;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                minus[r][x] = -__shfl_sync(0xffffffffu, lse, 4 * (2 * t + x)) * 1.4426950408889634f;
                limit[r][x] = __shfl_sync(0xffffffffu, lim, 4 * (2 * t + x));
            }
        }
        query_tile_f16<D, NR>(qrow, live, p.sm_log2, qb, qscale);
    }
    const int P = 1 << p.g.page_shift;
    const uint32_t* table =
        reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
    auto entry = [&](int jc) {
        const int j = jc + 16 * t;
        return jc < end && j < q.kv ? static_cast<int>(ldg_early(table + (j >> p.g.page_shift))) : 0;
    };
    int jc = j0 + warp * kFewChunk;
    int ahead = entry(jc);
    for (; jc < end; jc += kStride) {
        // (a block of 16 tokens behind the end, or on a bad page: page 0 is read; tokens behind the end are cut off, with a bad
        // page the results are void)
        const int blk = jc + 16 * t;
        const uint32_t mine = static_cast<uint32_t>(blk < q.kv && check_page(p.g, ahead) ? ahead : 0);
        const size_t kph = static_cast<size_t>(__shfl_sync(0xffffffffu, mine, g >> 1)) * p.g.kv_heads + h;
        const int kblk = jc + 16 * (g >> 1), koff = kblk & (P - 1);
        const uint8_t* kp = p.g.kcodes + (kph * P + koff + 2 * (g & 1)) * D + 16 * t;
        // m tile i of S^T: its row g is token kblk + 4 i + 2 (g & 1), its row g + 8 the next one
        uint4 kw[4][2][CH];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < CH; ++c) kw[i][x][c] = ldg_nc_na_v4(kp + (4 * i + x) * D + 64 * c);
        const uint4 ksw = ldg_nc_na_v4(p.g.kscale + kph * P + koff);
        const int j = kblk + 4 * t + 2 * (g & 1);  // the lane's tokens in the end: j, j + 1
        float2 old = make_float2(0.f, 0.f);
        if (j < stop) old.x = __ldcg(p.scores + at + j);
        if (j + 1 < stop) old.y = __ldcg(p.scores + at + j + 1);
        ahead = entry(jc + kStride);
        const uint32_t ks[4] = {ksw.x, ksw.y, ksw.z, ksw.w};
        float v[4][2];  // tokens kblk + 4 i + 2 (g & 1) + a: sums over the lane's rows
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float sc[NR][4];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[r][k] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint32_t wa[4] = {kw[i][0][c].x, kw[i][0][c].y, kw[i][0][c].z, kw[i][0][c].w};
                const uint32_t wb[4] = {kw[i][1][c].x, kw[i][1][c].y, kw[i][1][c].z, kw[i][1][c].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t x[4];
                    codes_f16(wa[k], x[0], x[2]);
                    codes_f16(wb[k], x[1], x[3]);
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(sc[r], x, qb[r][c * 4 + k][0], qb[r][c * 4 + k][1]);
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const float f = e8m0_float(ks[i] >> (16 * (g & 1)), a);
                const int token = kblk + 4 * i + 2 * (g & 1) + a;
                v[i][a] = 0.f;
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float w = ex2(fmaf(sc[r][2 * a + x] * f, qscale[r][x], minus[r][x]));
                        v[i][a] += token < limit[r][x] ? w : 0.f;
                    }
            }
        }
        // over the four lanes t, by halves of what is left: lane t ends with m tile t
        float u[2][2], z[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const bool up = (t & 2) != 0;
                const float keep = up ? v[2 + i][a] : v[i][a], give = up ? v[i][a] : v[2 + i][a];
                u[i][a] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
            }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const bool up = (t & 1) != 0;
            const float keep = up ? u[1][a] : u[0][a], give = up ? u[0][a] : u[1][a];
            z[a] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
        }
        if (j < stop) p.out[at + j] = j < q.kv ? old.x + z[0] : old.x;
        if (j + 1 < stop) p.out[at + j + 1] = j + 1 < q.kv ? old.y + z[1] : old.y;
    }
    // the rest of the range (behind the last chunk that was written above)
    const int done = end > j0 ? j0 + (end - j0 + kFewChunk - 1) / kFewChunk * kFewChunk : j0;
    for (int j = done + threadIdx.x; j < stop; j += kScoreWarps * 32) p.out[at + j] = p.scores[at + j];
}

template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) paged_scores_rows_kernel(PagedScoreParams p) {
    constexpr int CH = D / 64;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, s = blockIdx.z;
    const int j0 = (blockIdx.x * kScoreWarps + warp) * kScoreTokens;
    if (j0 >= p.g.max_kv) return;
    const Seq q = load_seq(p.g, s);
    const int64_t at = (static_cast<int64_t>(s) * p.g.kv_heads + h) * p.score_stride + j0;
    const int rows = q.n * p.group;
    float sum[4][2];
#pragma unroll
    for (int n = 0; n < 4; ++n) sum[n][0] = sum[n][1] = 0.f;
    // the first new token that sees token j0 or one before it
    const int first_new = p.causal ? max(0, j0 - (q.kv - q.n)) : 0;
    if (j0 < q.kv && rows > 0) {
        const int P = 1 << p.g.page_shift;
        uint32_t kb[4][CH * 4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n) {  // token j0 + 8 n + g
            const int j = j0 + 8 * n + g;
            const int page = j < q.kv ? load_page(p.g, s, j >> p.g.page_shift) : -1;
            const size_t row = (static_cast<size_t>(max(page, 0)) * p.g.kv_heads + h) * P + (j & (P - 1));
            const uint32_t f = page >= 0 ? scale_factor(__ldg(p.g.kscale + row)) : 0u;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint4 v = ldg_nc_na_v4(p.g.kcodes + row * D + 16 * (t + 4 * c));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kb[n][c * 4 + i][0] = bf2_mul(codes02(w[i]), f);
                    kb[n][c * 4 + i][1] = bf2_mul(codes13(w[i]), f);
                }
            }
        }
        for (int r0 = first_new * p.group; r0 < rows; r0 += 16) {
            uint32_t qa[CH * 4][4];
            float minus[2];
            int limit[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int rr = r0 + g + 8 * r;
                const bool live = rr < rows;
                const int tok = live ? rr / p.group : 0, head = h * p.group + (live ? rr - tok * p.group : 0);
                const __nv_bfloat16* qrow =
                    p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D;
                const float lse = live ? __ldg(p.lse + static_cast<int64_t>(q.q0 + tok) * p.heads + head) : -INFINITY;
                minus[r] = -lse * 1.4426950408889634f;
                limit[r] = lse == -INFINITY ? 0 : p.causal ? q.kv - q.n + tok + 1 : q.kv;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint4 a = __ldg(reinterpret_cast<const uint4*>(qrow + 16 * (t + 4 * c)));
                    const uint4 b = __ldg(reinterpret_cast<const uint4*>(qrow + 16 * (t + 4 * c) + 8));
                    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        qa[c * 4 + i][r] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
                        qa[c * 4 + i][2 + r] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < CH * 4; ++k) mma_bf16(sc, qa[k], kb[n][k][0], kb[n][k][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + 8 * n + 2 * t + (i & 1), r = i >> 1;
                    const float w = ex2(fmaf(sc[i], p.sm_log2, minus[r]));
                    sum[n][i & 1] += j < limit[r] ? w : 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float v = sum[n][b];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            sum[n][b] = v;
        }
    // lane (g, t): token 8 g + 2 t + {0, 1} for g < 4
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n)
        if (g == n) {
            a = sum[n][0];
            b = sum[n][1];
        }
    const int j = 8 * g + 2 * t;
    const int end = rows > 0 ? q.kv : 0;  // tokens from here on keep their scores
    if (g < 4 && j0 + j < p.g.max_kv) p.out[at + j] = j0 + j < end ? p.scores[at + j] + a : p.scores[at + j];
    if (g < 4 && j0 + j + 1 < p.g.max_kv) p.out[at + j + 1] = j0 + j + 1 < end ? p.scores[at + j + 1] + b : p.scores[at + j + 1];
}

template <int D>
cudaError_t launch_d(const PagedScoreParams& p, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    if (rows <= 16) {
        // Up to 16 rows stay in registers (8 KV heads x 128, 32 sequences of 8,000
        // tokens: 8 rows 45 us, 123 us with the kernel for some tiles; 16 rows 55
        // and 127).  Ranges of the
        // cached tokens: twelve blocks an SM, a step of every warp at least (16
        // sequences of 509 to 8,191 tokens x 8 heads: 6 blocks an SM 21.6 us, 12
        // 19.5, 24 21.8, 48 20.6)
        const int step = kScoreWarps * kFewChunk;
        const int64_t steps = (p.g.max_kv + step - 1) / step, lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
        const int64_t want = std::min(steps, std::max<int64_t>(1, (152 * 12 + lists - 1) / lists));
        const int range = static_cast<int>((steps + want - 1) / want) * step;
        const dim3 grid((p.g.max_kv + range - 1) / range, p.g.kv_heads, p.g.seqs);
        if (rows <= 8)
            paged_scores_few_kernel<D, 1><<<grid, kScoreWarps * 32, 0, s>>>(p, range);
        else
            paged_scores_few_kernel<D, 2><<<grid, kScoreWarps * 32, 0, s>>>(p, range);
        return cudaGetLastError();
    }
    const int per = kScoreWarps * kScoreTokens;
    dim3 grid((p.g.max_kv + per - 1) / per, p.g.kv_heads, p.g.seqs);
    paged_scores_rows_kernel<D><<<grid, kScoreWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_scores(const PagedScoreParams& p, int D, cudaStream_t s) {
    // Up to two row tiles of 16, while there is not much to read, the kernels here
    // are done before the tcgen05 kernel has set itself up (8 KV heads x 128, 32
    // rows: one sequence of 300 tokens 4.5 against 7.7 us, 8,000 tokens 8.9
    // against 10.3, 64 sequences of 300 19 against 34); then its conversion of K
    // keeps up better (one sequence of 60,000 tokens 41 against 33, 32 sequences
    // of 8,000 162 against 145; 16 of 1,000 14.5 against 15.1).  With more rows each
    // tile costs another pass here (one sequence of 8,000, 64 rows: 12.8 against
    // 10.6; 32 of 8,000, 128 rows: 401 against 146).
    const int64_t lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    const bool much = p.g.max_kv > 4096 && lists * p.g.max_kv > (1 << 17);
    if (rows > 16 && (rows > kScoreRowsMax || much)) return launch_paged_scores_tc(p, D, s);
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
