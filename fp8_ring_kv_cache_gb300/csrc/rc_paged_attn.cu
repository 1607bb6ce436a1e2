// rc_paged_attn.cu -- attention of each sequence's new tokens over its pages.
//
// paged_rows_kernel, for few query rows (a KV head's rows are its sequence's
// new tokens x the query heads that share it): bound by reading the codes, so
// the warps read them straight into the registers where the matrix
// instructions want them, with no shared memory and no barrier on the way.
// A block has one (sequence, KV head, split of the cached tokens) and all its rows, 8
// or 16 at most; a warp takes 64 cached tokens at a time, transposed, so that the few
// rows are the short side of the products (m16n8k16):
//   S^T = K Q^T  in fp16: one conversion makes two codes exact fp16 numbers, the
//                rows of Q are scaled to fp16's range, and the tokens' scales
//                (powers of two) multiply S.  A 16-byte piece of a K row is 16 of
//                the summed dims for its token; which dims of the product they
//                are is free as long as Q is held in the same order
//   P = exp2(S - max), online; an 8 x 8 transpose of the accumulators makes them
//                the B operand of
//   O^T += V^T P^T  in bf16, whose A operand is a 16-byte piece of a V row: 16
//                tokens of one dim, with their scales (which fp16 could not
//                hold).  The tokens of S's rows are chosen to match.  P is rounded
//                to bf16 for it (the row sums are not): at most 2^-8 of each weight
//                beside the 2^-8 of the bf16 result.
// Rows first (S = Q K^T) took twice the products and as many moves to keep the
// unused half of the accumulators in place: 134 us for 32 single tokens
// (sequences of 61 to 16,381 tokens, 8 KV heads x 6 query heads x 128), which
// now take 98.5 us: 544 MB, 0.81 of the rate of a copy.  The rest is the start
// and end of the blocks, and warps that hold too much to be more on an SM.
// The warps' (max, sum, O) are joined through shared memory; with several
// splits they go to the workspace, and the block that arrives last at its counter
// joins them in split order, so results do not depend on timing.
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr int kChunk = 64;      // cached tokens of a warp's step
constexpr int kMaxSplits = 32;  // of a sequence

// One split's result for 8 NR rows in the workspace: O [rows][D],
// then max and sum [rows] each.
template <int D, int NR>
constexpr int part_floats() {
    return 8 * NR * D + 2 * 8 * NR;
}

// Weight of a partial whose running max is m against the joint max M (both in
// log2 units; -inf: the partial saw nothing).
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }

// 8 NR rows (NR 1 or 2).
template <int D, int NR>
__global__ void __launch_bounds__(kRowsThreads, NR == 1 ? 3 : 2) paged_rows_kernel(PagedAttnParams p) {
    constexpr int kRowTile = 8 * NR;
    constexpr int CH = D / 64;  // 16-byte pieces of a K row that a lane reads
    constexpr int MT = D / 16;  // m tiles of O^T
    __shared__ __align__(16) float so[kRowsWarps][kRowTile][D + 4];
    __shared__ float sm[kRowsWarps][kRowTile], sl[kRowsWarps][kRowTile];
    __shared__ int last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
    const Seq q = load_seq(p.g, s);
    const int rows = q.n * p.group;  // at most kRowTile, as max_new new tokens have
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
        query_tile_f16<D, NR>(qrow, live, p.sm_log2, qb, qscale);
    }
    // what every row sees
    const int least = min(j1, p.causal ? max(0, q.kv - q.n + 1) : q.kv);

    float o[NR][MT][4];
    float m_run[NR][2], l_run[NR][2];
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
    const uint32_t* table =
        reinterpret_cast<const uint32_t*>(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages);
    auto entry = [&](int jc) {
        const int j = jc + 16 * t;
        return jc < j1 && j < q.kv ? static_cast<int>(ldg_early(table + (j >> p.g.page_shift))) : 0;
    };
    constexpr int kStride = kRowsWarps * kChunk;
    int ahead = entry(j0 + warp * kChunk);
    for (int jc = j0 + warp * kChunk; jc < j1; jc += kStride) {
        // The lane reads K rows and scales of the 16-token block g >> 1 and V
        // pieces and scales of block t.  A block behind the sequence's end, or on
        // a bad page, is read from page 0 instead, and its tokens are cut off (K)
        // or given the factor 0 (V).
        const int vblk = jc + 16 * t, kblk = jc + 16 * (g >> 1);
        const bool vok = vblk < q.kv && check_page(p.g, ahead);
        const uint32_t mine = static_cast<uint32_t>(vok ? ahead : 0);
        const size_t vph = static_cast<size_t>(mine) * p.g.kv_heads + h;
        const size_t kph = static_cast<size_t>(__shfl_sync(0xffffffffu, mine, g >> 1)) * p.g.kv_heads + h;
        const int koff = kblk & (P - 1), voff = vblk & (P - 1);
        const uint8_t* kp = p.g.kcodes + (kph * P + koff + 2 * (g & 1)) * D + 16 * t;
        const uint8_t* vp = p.g.vcodes + (vph * D + g) * P + voff;
        ahead = entry(jc + kStride);

        // m tile i of S^T: its row g is token kblk + 4 i + 2 (g & 1), its row g + 8 the next one
        uint4 kw[4][2][CH];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int c = 0; c < CH; ++c) kw[i][x][c] = ldg_nc_na_v4(kp + (4 * i + x) * D + 64 * c);
        const uint4 ksw = ldg_nc_na_v4(p.g.kscale + kph * P + koff);
        const uint4 vsw = ldg_nc_na_v4(p.g.vscale + vph * P + voff);
        // the first half of the V pieces is on its way while S is computed, the
        // second while the softmax runs
        uint4 vw[MT][2];
#pragma unroll
        for (int n = 0; n < MT / 2; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) vw[n][x] = ldg_nc_na_v4(vp + static_cast<size_t>(16 * n + 8 * x) * P);
        float sc[NR][4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[r][i][k] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint32_t wa[4] = {kw[i][0][c].x, kw[i][0][c].y, kw[i][0][c].z, kw[i][0][c].w};
                const uint32_t wb[4] = {kw[i][1][c].x, kw[i][1][c].y, kw[i][1][c].z, kw[i][1][c].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    codes_f16(wa[k], a[0], a[2]);
                    codes_f16(wb[k], a[1], a[3]);
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(sc[r][i], a, qb[r][c * 4 + k][0], qb[r][c * 4 + k][1]);
                }
            }
        }
#pragma unroll
        for (int n = MT / 2; n < MT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) vw[n][x] = ldg_nc_na_v4(vp + static_cast<size_t>(16 * n + 8 * x) * P);

        // softmax: scores 2 a + x of m tile i: token kblk + 4 i + 2 (g & 1) + a, row 2 t + x
        const bool full = jc + kChunk <= least;
        const uint32_t ks[4] = {ksw.x, ksw.y, ksw.z, ksw.w};
        float mx[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) mx[r][0] = mx[r][1] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const float f = e8m0_float(ks[i] >> (16 * (g & 1)), a);
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int x = 0; x < 2; ++x) sc[r][i][2 * a + x] *= f;
            }
        if (!full) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int j = kblk + 4 * i + 2 * (g & 1) + a;
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            if (j >= limit[r][x] || j >= j1) sc[r][i][2 * a + x] = -INFINITY;
                }
        }
        bool moved = false;
        float base[NR][2], alpha[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[r][x] = max3(mx[r][x], sc[r][i][x], sc[r][i][2 + x]);
                mx[r][x] = fmaxf(mx[r][x], __shfl_xor_sync(0xffffffffu, mx[r][x], 4));
                mx[r][x] = fmaxf(mx[r][x], __shfl_xor_sync(0xffffffffu, mx[r][x], 8));
                mx[r][x] = fmaxf(mx[r][x], __shfl_xor_sync(0xffffffffu, mx[r][x], 16));
                const float m_new = fmaxf(m_run[r][x], mx[r][x] * qscale[r][x]);
                base[r][x] = m_new == -INFINITY ? 0.f : m_new;
                alpha[r][x] = ex2(m_run[r][x] - base[r][x]);  // 0 while nothing was seen
                m_run[r][x] = m_new;
                moved |= alpha[r][x] != 1.f;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        const float w = ex2(fmaf(sc[r][i][2 * a + x], qscale[r][x], -base[r][x]));
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
        // the V pieces' 16 tokens: factors by word
        uint32_t vf[8];
        const uint32_t vs[4] = {vsw.x, vsw.y, vsw.z, vsw.w};
        uint32_t nans = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nans |= __vcmpgtu4(vs[i], 0x86868686u);
            vf[2 * i] = factors02(vs[i]);
            vf[2 * i + 1] = factors13(vs[i]);
        }
        if (!full || __any_sync(0xffffffffu, nans != 0 || !vok)) {
            // factor 0 for tokens the sequence does not have.  A token whose V is
            // not a number must reach the rows that see it and no other, so that
            // is moved from V (0 x NaN would reach every row) into the weights.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t good = vs[i] & ~__vcmpgtu4(vs[i], 0x86868686u);
                const int left = vok ? q.kv - (vblk + 4 * i) : 0;  // tokens of the word that exist
                vf[2 * i] = factors02(good) & ((left > 0 ? 0xffffu : 0u) | (left > 2 ? 0xffff0000u : 0u));
                vf[2 * i + 1] = factors13(good) & ((left > 1 ? 0xffffu : 0u) | (left > 3 ? 0xffff0000u : 0u));
                // the scores' tokens are of block g >> 1, which lane g >> 1 has the scales of
                const uint32_t theirs = __shfl_sync(0xffffffffu, vs[i], g >> 1);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    const int j = kblk + 4 * i + 2 * (g & 1) + a;
                    if (((theirs >> (8 * (2 * (g & 1) + a))) & 0xffu) > 134u) {
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (j < limit[r][x] && j < j1) sc[r][i][2 * a + x] = __uint_as_float(0x7fc00000u);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // products over tokens 16 t + 4 i + {0, 2} and + {1, 3} of the chunk
            uint32_t pb[NR][2];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int a = 0; a < 2; ++a) pb[r][a] = transpose8(pack_bf16(sc[r][i][2 * a], sc[r][i][2 * a + 1]));
#pragma unroll
            for (int n = 0; n < MT; ++n) {
                uint32_t a[4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t w = i == 0 ? vw[n][x].x : i == 1 ? vw[n][x].y : i == 2 ? vw[n][x].z : vw[n][x].w;
                    a[x] = bf2_mul(codes02(w), vf[2 * i]);
                    a[2 + x] = bf2_mul(codes13(w), vf[2 * i + 1]);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) mma_bf16(o[r][n], a, pb[r][0], pb[r][1]);
            }
        }
    }

    // ---- join the warps
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
                sm[warp][row] = m_run[r][x];
                sl[warp][row] = l;
            }
#pragma unroll
            for (int n = 0; n < MT; ++n) {
                so[warp][row][16 * n + g] = o[r][n][x];
                so[warp][row][16 * n + 8 + g] = o[r][n][2 + x];
            }
        }
    __syncthreads();
    const int slot = s * p.g.kv_heads + h;
    float* part = p.part + static_cast<size_t>(slot) * p.splits * part_floats<D, NR>();
    auto store_out = [&](int r, int d, float4 v, float M, float L) {
        const int tok = r / p.group, head = h * p.group + r - tok * p.group;
        const float inv = L > 0.f || L != L ? 1.f / L : 0.f;  // a sum that is not a number stays one
        *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(q.q0 + tok) * p.out_stride +
                                  static_cast<int64_t>(head) * D + d) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
        if (d == 0 && p.lse != nullptr)
            p.lse[static_cast<int64_t>(q.q0 + tok) * p.heads + head] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    for (int i = tid; i < rows * (D / 4); i += kRowsThreads) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sm[w][r]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) {
            const float f = join_weight(sm[w][r], M);
            const float4 v = *reinterpret_cast<const float4*>(&so[w][r][d]);
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
            L += f * sl[w][r];
        }
        if (nsplit == 1) {
            store_out(r, d, acc, M, L);
        } else {
            float* mine = part + static_cast<size_t>(split) * part_floats<D, NR>();
            *reinterpret_cast<float4*>(mine + r * D + d) = acc;
            if (d == 0) {
                mine[kRowTile * D + r] = M;
                mine[kRowTile * D + kRowTile + r] = L;
            }
        }
    }
    if (nsplit == 1) return;
    // ---- join the splits: the last block to arrive
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(p.counters + slot, 1) == nsplit - 1;
    __syncthreads();
    if (!last) return;
    if (tid == 0) p.counters[slot] = 0;
    __threadfence();
    // the splits' weights first, some lanes a row; then O with many loads on the way
    constexpr int kLanes = kRowsThreads / kRowTile;  // of a row: 8 or 16, in one warp
    constexpr int kBatch = 16;                       // loads on the way
    static_assert(kMaxSplits % kBatch == 0 && kMaxSplits % kLanes == 0, "weights up to the last batch's end");
    static_assert(kRowsWarps * (D + 4) >= kMaxSplits, "the weights fit where the warps' O was");
    float* weight = &so[0][0][0];  // [split][row]
    {
        const int r = tid / kLanes, k0 = tid % kLanes;
        constexpr int K = kMaxSplits / kLanes;
        float m[K], l[K], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = k0 + i * kLanes;
            const float* b = part + static_cast<size_t>(k) * part_floats<D, NR>() + kRowTile * D + r;
            const bool have = k < nsplit && r < rows;
            m[i] = have ? __ldcg(b) : -INFINITY;
            l[i] = have ? __ldcg(b + kRowTile) : 0.f;
            M = fmaxf(M, m[i]);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float f = join_weight(m[i], M);
            L += f * l[i];
            weight[(k0 + i * kLanes) * kRowTile + r] = f;
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
        if (k0 == 0) {
            sm[0][r] = M;
            sl[0][r] = L;
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += kRowsThreads) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* from = part + r * D + d;
        for (int k0 = 0; k0 < nsplit; k0 += kBatch) {
            float4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                v[u] = k0 + u < nsplit ? __ldcg(reinterpret_cast<const float4*>(
                                             from + static_cast<size_t>(k0 + u) * part_floats<D, NR>()))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float f = weight[(k0 + u) * kRowTile + r];  // 0 behind the last split
                acc.x += f * v[u].x;
                acc.y += f * v[u].y;
                acc.z += f * v[u].z;
                acc.w += f * v[u].w;
            }
        }
        store_out(r, d, acc, sm[0][r], sl[0][r]);
    }
}

template <int D, int NR>
cudaError_t launch_rows(PagedAttnParams& p, size_t part_floats_max, int max_counters, cudaStream_t s) {
    const int64_t slots = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    // Splits: sixteen blocks an SM, which evens out sequences of different
    // lengths (8 query heads' groups of 6 x 32 sequences of 61 to 16,381 tokens:
    // 6 blocks an SM 119 us, 12 102, 16 99, 24 101, 48 106), at most 32, which
    // the last block can still join quickly, and as many as the workspace holds.
    // A block takes two steps of every warp at least (64 sequences x 1,000
    // tokens x 8 heads: one step 41 us, two 37), or one while each block has an
    // SM, or half of one with 8 rows, to itself (one sequence of 4,000 tokens:
    // one step 8.6 us, two 11.1; with 16 rows 11.0 and 13.6; 8,000 tokens with
    // 16 rows 15.5 and 13.6).  512 tokens stay whole (337 tokens: 6.5 us, as two
    // splits 7.8).
    const int step = kRowsWarps * kChunk;
    const int64_t steps = (p.g.max_kv + step - 1) / step;
    int64_t want = std::min<int64_t>((152 * 16 + slots - 1) / slots, kMaxSplits);
    const int least = steps > 2 && std::min<int64_t>(steps, kMaxSplits) * slots <= (NR == 1 ? 2 : 1) * 152 ? 1 : 2;
    want = std::min<int64_t>(want, (steps + least - 1) / least);
    want = std::min<int64_t>(want, static_cast<int64_t>(part_floats_max / (slots * part_floats<D, NR>())));
    if (slots > max_counters || want < 1) want = 1;
    const int per = static_cast<int>((p.g.max_kv + want - 1) / want);
    p.split_tokens = std::max(step, (per + step - 1) / step * step);
    p.splits = std::max(1, (p.g.max_kv + p.split_tokens - 1) / p.split_tokens);
    dim3 grid(p.splits, p.g.kv_heads, p.g.seqs);
    paged_rows_kernel<D, NR><<<grid, kRowsThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_attention_d(PagedAttnParams& p, size_t part_floats_max, int max_counters, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    // Up to 16 rows per KV head the reading of the codes is what counts; with
    // more, each tile of 16 would read them again, and the tcgen05 kernel, whose
    // time hardly grows up to 128 rows, is the faster one (32 sequences x 8,000
    // tokens x 8 KV heads x 128: 8 rows 97 against 245 us, 16 rows 122 against
    // 245).  Tiles of 8 rows save half the products (the same with 1 row: 95 us as
    // a tile of 8, 124 us as one of 16).
    if (rows <= 8) return launch_rows<D, 1>(p, part_floats_max, max_counters, s);
    if (rows <= 16) return launch_rows<D, 2>(p, part_floats_max, max_counters, s);
    return launch_paged_tc(p, D, part_floats_max, s);
}

}  // namespace

cudaError_t launch_paged_attention(PagedAttnParams& p, int D, size_t part_floats_max, int max_counters,
                                   cudaStream_t s) {
    return D == 128 ? launch_attention_d<128>(p, part_floats_max, max_counters, s)
                    : launch_attention_d<64>(p, part_floats_max, max_counters, s);
}

}  // namespace rc
