// rc_paged4_attn.cu -- attention of few query rows over the 4-bit pages.
//
// Bound by reading the codes, so the warps read them straight into the registers
// where the matrix instructions want them.  A block has one (sequence, KV head,
// split of the cached tokens) and all its rows, 8 or 16 at most; a warp takes 64
// cached tokens at a time, transposed, so that the few rows are the short side of
// the products (m16n8k16, fp16 operands, fp32 sums):
//   S^T = K Q^T      a lane's 16 bytes of a K row are 32 of the summed dims for its
//                    token; which dims of a product they are is free as long as Q is
//                    held in the same order.  Rows of Q are scaled to fp16's range.
//   P = exp2(S - max + 14), online, rounded to fp16 (2^-12 of each weight; weights down
//                    to 2^-28 of the largest keep all their bits, the row sums are
//                    not rounded); an 8 x 8 transpose of the accumulators makes them
//                    the B operand of
//   O^T += V^T P^T   whose A operand is an 8-byte piece of a V row: 16 tokens of one dim.
//                    The tokens of S's rows are chosen to match.
// One conversion makes two codes exact fp16 numbers and one multiplication scales
// them, exactly: a code times a scale has 6 bits.  A scale byte is an fp16 number but
// for a shift.  The scales of K come with the lane's dims; a lane reads those of V of one
// block of 16 dims for its 16 tokens, and the lanes hand them to one another.
#include "rc_paged4.cuh"
#include "rc_paged_rows.cuh"

namespace rc {

namespace {

constexpr float kWeightShift = 14.f;  // log2 of the largest weight in fp16

__device__ __forceinline__ uint2 ldg_nc_na_v2(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// 8 NR rows (NR 1 or 2).
template <int D, int NR>
__global__ void __launch_bounds__(kRowsThreads, NR == 1 ? 3 : 2) paged4_rows_kernel(PagedAttnParams p) {
    constexpr int KW = D / 32;  // words of a K row that a lane reads
    constexpr int KB = D / 64;  // blocks of 16 dims among them
    constexpr int MT = D / 16;  // m tiles of O^T: blocks of 16 dims
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
    const Seq q = load_seq(p.g, s);
    const int rows = q.n * p.group;  // at most 8 NR, as max_new new tokens have
    if (rows == 0) return;
    const int nsplit = max(1, (q.kv + p.split_tokens - 1) / p.split_tokens);  // (the last row sees every token)
    if (split >= nsplit) return;
    const int j0 = split * p.split_tokens, j1 = min(q.kv, j0 + p.split_tokens);

    uint32_t qb[NR][D / 16][2];
    float qscale[NR][2];
    // of the rows 2 t + x of each eight, whose scores the lane gets: tokens seen
    // (rows past the end see all; nothing of theirs is stored)
    int limit[NR][2];
    {
        const __nv_bfloat16* qrow[NR];
        bool live[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int rr = 8 * r + g;
            live[r] = rr < rows;
            const int tok = live[r] ? rr / p.group : 0, head = h * p.group + (live[r] ? rr - tok * p.group : 0);
            qrow[r] = p.q + static_cast<int64_t>(q.q0 + tok) * p.q_stride + static_cast<int64_t>(head) * D;
            const int lim = !live[r] ? 1 << 30 : p.causal ? max(0, q.kv - q.n + tok + 1) : q.kv;
#pragma unroll
            for (int x = 0; x < 2; ++x) limit[r][x] = __shfl_sync(0xffffffffu, lim, 4 * (2 * t + x));
        }
        query_tile_f16<D, NR, D / 4>(qrow, live, p.sm_log2, qb, qscale);
    }
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
    const int P = 1 << p.g.page_shift;
    // Lane l < 4 of each four reads the page of the chunk's block l of 16 tokens a
    // chunk ahead.
    const uint32_t* pages =
        reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
    auto entry = [&](int jc) {
        const int j = jc + 16 * t;
        return jc < j1 && j < q.kv ? static_cast<int>(ldg_early(pages + (j >> p.g.page_shift))) : 0;
    };
    constexpr int kStride = kRowsWarps * kChunk;
    int ahead = entry(j0 + warp * kChunk);
    for (int jc = j0 + warp * kChunk; jc < j1; jc += kStride) {
        // The lane reads K rows and scales of the 16-token block g >> 1 and V
        // pieces and scales of block t.  A block behind the sequence's end, or on
        // a bad page, is read from page 0 instead, and its tokens are cut off (K)
        // or given the scale 0 (V).
        const int vblk = jc + 16 * t, kblk = jc + 16 * (g >> 1);
        const bool vok = vblk < q.kv && check_page(p.g, ahead);
        const uint32_t mine = static_cast<uint32_t>(vok ? ahead : 0);
        const size_t vph = static_cast<size_t>(mine) * p.g.kv_heads + h;
        const size_t kph = static_cast<size_t>(__shfl_sync(0xffffffffu, mine, g >> 1)) * p.g.kv_heads + h;
        const int koff = kblk & (P - 1), voff = vblk & (P - 1);
        const uint8_t* kp = p.g.kcodes + (kph * P + koff + (g & 1)) * (D / 2) + t * (D / 8);
        const uint8_t* vp = p.g.vcodes + ((vph * D + g) * P + voff) / 2;
        ahead = entry(jc + kStride);

        // m tile i of S^T: its row g is token kblk + 4 i + (g & 1), its row g + 8 the next but one
        uint32_t kw[4][2][KW];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint8_t* from = kp + (4 * i + 2 * x) * (D / 2);
                if constexpr (KW == 4) {
                    const uint4 w = ldg_nc_na_v4(from);
                    kw[i][x][0] = w.x, kw[i][x][1] = w.y, kw[i][x][2] = w.z, kw[i][x][3] = w.w;
                } else {
                    const uint2 w = ldg_nc_na_v2(from);
                    kw[i][x][0] = w.x, kw[i][x][1] = w.y;
                }
            }
        uint4 ksw[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) ksw[b] = ldg_nc_na_v4(p.g.kscale + (kph * MT + KB * t + b) * P + koff);
        // block g of V's dims
        const uint4 vsw = ldg_nc_na_v4(p.g.vscale + (vph * MT + (g & (MT - 1))) * P + voff);
        uint2 vw[MT][2];
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) vw[n][x] = ldg_nc_na_v2(vp + static_cast<size_t>(16 * n + 8 * x) * (P / 2));
        float sc[NR][4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[r][i][k] = 0.f;
            uint32_t f[2][KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const uint32_t w = i == 0 ? ksw[b].x : i == 1 ? ksw[b].y : i == 2 ? ksw[b].z : ksw[b].w;
                f[0][b] = scale_twice(w, g & 1);
                f[1][b] = scale_twice(w, 2 + (g & 1));
            }
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                uint32_t wa[4], wb[4];
                codes8_f16(kw[i][0][k], wa);
                codes8_f16(kw[i][1][k], wb);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t a[4] = {half2_mul(wa[2 * c], f[0][k / 2]), half2_mul(wb[2 * c], f[1][k / 2]),
                                           half2_mul(wa[2 * c + 1], f[0][k / 2]), half2_mul(wb[2 * c + 1], f[1][k / 2])};
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(sc[r][i], a, qb[r][2 * k + c][0], qb[r][2 * k + c][1]);
                }
            }
        }

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
                const float m_new = fmaxf(m_run[r][x], mx * qscale[r][x] - kWeightShift);
                const float base = m_new == -INFINITY ? 0.f : m_new;
                alpha[r][x] = ex2(m_run[r][x] - base);  // 0 while nothing was seen
                m_run[r][x] = m_new;
                moved |= alpha[r][x] != 1.f;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float w = ex2(fmaf(sc[r][i][2 * a + x], qscale[r][x], -base));
                        sc[r][i][2 * a + x] = w;
                        sum += w;
                    }
                l_run[r][x] = l_run[r][x] * alpha[r][x] + sum;
            }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int n = 0; n < MT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][n][i] *= alpha[r][i & 1];
        }
        uint32_t vs[4] = {vsw.x, vsw.y, vsw.z, vsw.w};
        uint32_t nans = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) nans |= __vcmpgtu4(vs[i], 0x01010101u * (kFirstNan4 - 1));
        if (!full || __any_sync(0xffffffffu, nans != 0 || !vok)) {
            // scale 0 for tokens the sequence does not have.  A token whose V is not a
            // number (its first block says so) must reach the rows that see it and no
            // other, so that is moved from V (0 x NaN would reach every row) into the
            // weights.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the scores' tokens are of block g >> 1, which lane g >> 1 has the first scales of
                const uint32_t theirs = __shfl_sync(0xffffffffu, vs[i], g >> 1);
                const int left = vok ? q.kv - (vblk + 4 * i) : 0;  // tokens of the word that exist
                const uint32_t have = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
                vs[i] &= have & ~__vcmpgtu4(vs[i], 0x01010101u * (kFirstNan4 - 1));
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int j = kblk + 4 * i + 2 * a + (g & 1);
                    if (((theirs >> (8 * (2 * a + (g & 1)))) & 0xffu) >= kFirstNan4) {
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (j < limit[r][x] && j < j1) sc[r][i][2 * a + x] = __uint_as_float(0x7fc00000u);
                    }
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
#pragma unroll
        for (int n = 0; n < MT; ++n) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint32_t lo[4], hi[4];
                codes8_f16(w ? vw[n][0].y : vw[n][0].x, lo);
                codes8_f16(w ? vw[n][1].y : vw[n][1].x, hi);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int i = 2 * w + c;
                    const uint32_t word = __shfl_sync(0xffffffffu, vs[i], 4 * n + t);
                    const uint32_t f0 = scales01(word), f1 = scales23(word);
                    const uint32_t a[4] = {half2_mul(lo[2 * c], f0), half2_mul(hi[2 * c], f0), half2_mul(lo[2 * c + 1], f1),
                                           half2_mul(hi[2 * c + 1], f1)};
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(o[r][n], a, pb[r][i][0], pb[r][i][1]);
                }
            }
        }
    }
    join_rows<D, NR>(p, q, s, h, split, nsplit, o, m_run, l_run);
}

template <int D, int NR>
cudaError_t launch_rows(PagedAttnParams& p, size_t part_floats_max, int max_counters, cudaStream_t s) {
    split_rows<D, NR>(p, part_floats_max, max_counters);
    dim3 grid(p.splits, p.g.kv_heads, p.g.seqs);
    paged4_rows_kernel<D, NR><<<grid, kRowsThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_attention_d(PagedAttnParams& p, size_t part_floats_max, int max_counters, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    if (rows <= 8) return launch_rows<D, 1>(p, part_floats_max, max_counters, s);
    if (rows <= 16) return launch_rows<D, 2>(p, part_floats_max, max_counters, s);
    return launch_paged4_tc(p, D, part_floats_max, s);
}

}  // namespace

cudaError_t launch_paged4_attention(PagedAttnParams& p, int D, size_t part_floats_max, int max_counters,
                                    cudaStream_t s) {
    return D == 128 ? launch_attention_d<128>(p, part_floats_max, max_counters, s)
                    : launch_attention_d<64>(p, part_floats_max, max_counters, s);
}

}  // namespace rc
