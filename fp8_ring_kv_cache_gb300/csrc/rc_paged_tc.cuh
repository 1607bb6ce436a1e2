// rc_paged_tc.cuh -- what the tcgen05 attention kernels over pages share: row tiles
// and how their cached tokens are split, the joining of the splits, the launch.
#pragma once
#include <algorithm>
#include <type_traits>

#include "rc_paged.cuh"

namespace rc {

// A launch of 640 threads has 96 registers a thread.
constexpr int kTcThreads = 640;
constexpr int kTileM = 128, kTileN = 128;
constexpr int kRowsTc = 2 * kTileM;
static_assert(kRowsTc == kAttendRows, "the blocks that the host counts");
constexpr int kWgSoftmax0 = 1, kWgConvertK = 3;
constexpr uint32_t kTcTmem = 512;

// A split's result for a row tile: O [256][D] (joined weights, not divided),
// then max and sum [256] each.
template <int D>
constexpr int tc_part_floats() {
    return kRowsTc * D + 2 * kRowsTc;
}

// The first `left` of 16 bytes, the others 0.
__device__ __forceinline__ uint4 cut16(uint4 v, int left) {
    auto cut = [](uint32_t w, int n) { return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u); };
    return make_uint4(cut(v.x, left), cut(v.y, left - 4), cut(v.z, left - 8), cut(v.w, left - 12));
}

// Cached tokens that the rows of a tile see, and how they are split.
struct TileWork {
    int rows;    // rows of the sequence's KV head (0: none, or another kernel's)
    int seen;    // tokens that the tile's last row sees
    int nsplit;  // splits with work (at least 1)
};
__device__ __forceinline__ TileWork tile_work(const PagedAttnParams& p, const Seq& q, int tile) {
    TileWork w;
    w.rows = q.n * p.group;
    if (w.rows <= p.few) w.rows = 0;
    const int last_new = min(q.n - 1, (tile * kRowsTc + kRowsTc - 1) / p.group);
    w.seen = p.causal ? max(0, q.kv - q.n + last_new + 1) : q.kv;
    w.nsplit = max(1, (w.seen + p.split_tokens - 1) / p.split_tokens);
    return w;
}

// Tile number `number` among the tiles of all sequences (each sequence's last one first): its sequence, or -1 if there are
// fewer.  By the whole block, with some of its shared memory.
__device__ __forceinline__ int tile_place(const PagedAttnParams& p, int number, int& tile, int* smem) {
    constexpr int kWarps = kTcThreads / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (p.g.seqs + kTcThreads - 1) / kTcThreads;
    const int first = min(p.g.seqs, tid * per), end = min(p.g.seqs, first + per);
    auto tiles_of = [&](int s) {
        const int rows = load_seq(p.g, s).n * p.group;
        return rows <= p.few ? 0 : (rows + kRowsTc - 1) / kRowsTc;
    };
    int mine = 0;
    for (int s = first; s < end; ++s) mine += tiles_of(s);
    int to = mine;  // up to and with the thread's, of the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += x;
    }
    if (lane == 31) smem[warp] = to;
    if (tid == 0) smem[kWarps] = -1;  // (lengths that contradict each other may leave the number to nobody)
    __syncthreads();
    int before = to - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int n = smem[w];
        if (w < warp) before += n;
        all += n;
    }
    if (number >= all) return -1;
    if (before <= number && number < before + mine) {  // one thread
        for (int s = first; s < end; ++s) {
            const int n = tiles_of(s);
            if (number < before + n) {
                smem[kWarps] = s;
                smem[kWarps + 1] = n - 1 - (number - before);
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    const int s = smem[kWarps];
    tile = smem[kWarps + 1];
    __syncthreads();
    return s;
}

// Joins the splits of each row, in split order: a warp a row.
template <int D>
__global__ void __launch_bounds__(256) paged_tc_join_kernel(PagedAttnParams p) {
    using Piece = std::conditional_t<D == 128, float4, float2>;  // of a row, a lane's
    const int lane = threadIdx.x & 31;
    int b = blockIdx.x;
    const int h = b % p.g.kv_heads;
    b /= p.g.kv_heads;
    const int s = b % p.g.seqs, row = (b / p.g.seqs) * 8 + (threadIdx.x >> 5);
    const Seq q = load_seq(p.g, s);
    const int tile = row / kRowsTc;
    const TileWork tw = tile_work(p, q, tile);
    if (row >= tw.rows || tw.nsplit == 1) return;
    const int tr = row - tile * kRowsTc;
    const int slot = (s * p.row_tiles + tile) * p.g.kv_heads + h;
    const float* part = p.part + static_cast<size_t>(slot) * p.splits * tc_part_floats<D>();
    const float* ml = part + kRowsTc * D + tr;
    float M = -INFINITY;
    for (int k = lane; k < tw.nsplit; k += 32) M = fmaxf(M, __ldg(ml + static_cast<size_t>(k) * tc_part_floats<D>()));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    constexpr int V = D / 32;
    constexpr int kBatch = 8;  // loads on the way
    float acc[V], L = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int k0 = 0; k0 < tw.nsplit; k0 += 32) {
        float f = 0.f;  // weight of split k0 + lane
        if (k0 + lane < tw.nsplit) {
            const float* mine = ml + static_cast<size_t>(k0 + lane) * tc_part_floats<D>();
            const float m = __ldg(mine);
            f = m == -INFINITY ? 0.f : ex2(m - M);
            L += f * __ldg(mine + kRowsTc);
        }
        const int here = min(32, tw.nsplit - k0);
        for (int k = 0; k < here; k += kBatch) {
            Piece v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int at = min(k + u, here - 1);  // (again the last one: its weight here is 0)
                v[u] = __ldg(reinterpret_cast<const Piece*>(part + static_cast<size_t>(k0 + at) * tc_part_floats<D>() +
                                                            static_cast<size_t>(tr) * D + V * lane));
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float fu = __shfl_sync(0xffffffffu, f, k + u);
                const float w = k + u < here ? fu : 0.f;
                const float* x = reinterpret_cast<const float*>(&v[u]);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += w * x[i];
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float inv = (L > 0.f || L != L) ? 1.f / L : 0.f;
    const int tok = row / p.group, head = h * p.group + row - tok * p.group;
    __nv_bfloat16* out = p.out + static_cast<int64_t>(q.q0 + tok) * p.out_stride + static_cast<int64_t>(head) * D + V * lane;
#pragma unroll
    for (int i = 0; i < V; i += 2)
        *reinterpret_cast<uint32_t*>(out + i) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(q.q0 + tok) * p.heads + head] =
            L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// A kernel, and the devices where its shared memory's limit is set.
struct TilesKernel {
    void (*kernel)(PagedAttnParams);
    std::atomic<uint64_t>& configured;
};

// numbered: the kernel whose blocks are numbered over the tiles that there are; only for p.few > 0.
template <int D>
cudaError_t launch_tiles(const TilesKernel& padded, const TilesKernel& numbered, uint32_t smem, PagedAttnParams& p, size_t part_floats_max,
                         cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.g.max_new) * p.group;
    p.row_tiles = static_cast<int>((rows + kRowsTc - 1) / kRowsTc);
    const int64_t blocks = paged_attend_blocks(p.g, rows);
    // Splits: while there are fewer blocks than SMs, down to four KV tiles
    // each (a block's set-up and the join take as long as a few tiles), as many
    // as the workspace holds.  One sequence of 8,000 tokens x 8 KV heads x 128
    // with 64 rows: 118 us whole, 21 us in 16 splits of four tiles, 26 in eight.
    int64_t want = std::max<int64_t>(1, 152 / blocks);
    want = std::min<int64_t>(want, (p.g.max_kv + 4 * kTileN - 1) / (4 * kTileN));
    want = std::min<int64_t>(want, static_cast<int64_t>(part_floats_max / (blocks * tc_part_floats<D>())));
    want = std::max<int64_t>(want, 1);
    const int per = static_cast<int>((p.g.max_kv + want - 1) / want);
    p.split_tokens = std::max(kTileN, (per + kTileN - 1) / kTileN * kTileN);
    p.splits = std::max(1, (p.g.max_kv + p.split_tokens - 1) / p.split_tokens);
    // Where short sequences are another kernel's, most places of the padded grid are empty: unsplit, a block finds its tile
    // by its number among those that there are.  So many at most: the whole ones of all tokens, and one of each sequence.
    // (63 single tokens and a chunk of 512 in one call, all with 8,000 cached, 8 x 6 heads x 128: 768 tiles of a KV head in
    // the padded grid, 286 us in all; 77 numbered ones, 222.)
    int64_t grid = blocks;
    const bool by_number = p.few > 0 && p.splits == 1;
    if (by_number) {
        const int64_t tokens = p.g.tokens, longer = std::min<int64_t>(p.g.seqs, tokens / (p.few / p.group + 1));
        grid = std::min(tokens * p.group / kRowsTc + longer, blocks / p.g.kv_heads) * p.g.kv_heads;
        if (grid == 0) return cudaSuccess;
    }
    const TilesKernel& k = by_number ? numbered : padded;
    cudaError_t e = smem_limit_once(k.kernel, smem, k.configured);
    if (e != cudaSuccess) return e;
    k.kernel<<<dim3(static_cast<unsigned>(grid), p.splits), kTcThreads, smem, s>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t joins = (rows + 7) / 8 * p.g.seqs * p.g.kv_heads;
    paged_tc_join_kernel<D><<<static_cast<unsigned>(joins), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rc
