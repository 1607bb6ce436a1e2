// rc_paged_rows.cuh -- what the attention kernels for few query rows share: the split
// of the cached tokens over blocks, and the joining of the warps' and the splits'
// results.
#pragma once
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

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

// Joins the warps' results of a block, and of a sequence's splits in the block that arrives last: O^T accumulators o[r][n]
// (dims 16 n + g and + 8, rows 8 r + 2 t and + 1, of lane 4 g + t), running maxima and the lane's parts of the sums.
template <int D, int NR>
__device__ __forceinline__ void join_rows(const PagedAttnParams& p, const Seq& q, int s, int h, int split, int nsplit,
                                          const float (&o)[NR][D / 16][4], const float (&m_run)[NR][2], const float (&l_run)[NR][2]) {
    constexpr int kRowTile = 8 * NR, MT = D / 16;
    __shared__ __align__(16) float so[kRowsWarps][kRowTile][D + 4];
    __shared__ float sm[kRowsWarps][kRowTile], sl[kRowsWarps][kRowTile];
    __shared__ int last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int rows = q.n * p.group;
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

// Splits of the cached tokens.
template <int D, int NR>
void split_rows(PagedAttnParams& p, size_t part_floats_max, int max_counters) {
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
}

}  // namespace rc
