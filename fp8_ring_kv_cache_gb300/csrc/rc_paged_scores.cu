// rc_paged_scores.cu -- the attention weight that each cached token received:
// out[j] = scores[j] + sum over the query rows of exp(q . k_j scale - lse).
//
// paged_scores_rows_kernel, for few query rows: bound by reading the K codes.
// A warp owns 32 cached tokens of one (sequence, KV head), decodes their K rows
// to bf16 once, into the registers where the matrix instructions want them, and
// goes over the head's query rows 16 at a time.  A token's sum stays with its
// owner, so no two threads add to one entry and the order is fixed.
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kScoreWarps = 4;
constexpr int kScoreTokens = 32;  // of a warp
constexpr int kScoreRowsMax = 128;

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
    if (g < 4 && j0 + j < p.g.max_kv) p.out[at + j] = p.scores[at + j] + a;
    if (g < 4 && j0 + j + 1 < p.g.max_kv) p.out[at + j + 1] = p.scores[at + j + 1] + b;
}

template <int D>
cudaError_t launch_d(const PagedScoreParams& p, cudaStream_t s) {
    const int per = kScoreWarps * kScoreTokens;
    dim3 grid((p.g.max_kv + per - 1) / per, p.g.kv_heads, p.g.seqs);
    paged_scores_rows_kernel<D><<<grid, kScoreWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_scores(const PagedScoreParams& p, int D, cudaStream_t s) {
    // up to a few row tiles the warps' own products keep up with the reading of
    // the codes; with more rows the tensor cores' do
    if (static_cast<int64_t>(p.g.max_new) * p.group > kScoreRowsMax) return launch_paged_scores_tc(p, D, s);
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
