// rc_paged_evict.cu -- cutting sequences to a budget by accumulated attention
// weight.
//
// paged_select_kernel: one block per (sequence, KV head) finds the budget's
//    threshold among the scores by radix selection, 11, 11 and 10 bits of the
//    ordered key a pass (the keys stay in shared memory while they fit; the
//    first pass then tells four sizes an octave apart, so that few lanes meet
//    in one counter), then lists the kept indices in ascending order: each warp
//    counts in its own run of scores with ballots, the counts are summed over
//    the warps, and each warp writes its run.  Ties at the threshold go to the
//    lowest index.
// paged_gather_kernel: copies the kept tokens to the new pages: bound by
//    memory.  K rows go 16 bytes a thread.  A V row has one byte per token: for
//    16 kept tokens at a time the 16-byte pieces that hold them (at most 16,
//    usually three or four) are brought to shared memory for every dim, the
//    bytes are picked there, and rows of 64 go out.  (Single bytes from and to
//    global memory, 32 tokens side by side, took 132 us for 64 lists of 8,192.)
//    K rows, scales and V's pieces are on their way together.
//
// 8 sequences of 9,001 to 32,749 tokens x 8 heads x 128, 8,192 of each kept: 95 us,
// 24 of them the selection (64 blocks, as many as there are lists; its passes over
// the keys follow one another) and 71 the copies: 350 MB at 4.9 TB/s, as the pieces
// of V are read with the tokens between those that stay.
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kBatch = 16;               // scores of a thread on their way
constexpr int kHistCopies = 2;           // histograms that even and odd lanes have to themselves
// Keys kept in shared memory (8 sequences of 32,749 tokens x 8 heads, 1,024 of
// each kept: 11 us less than when every pass reads the scores again).
constexpr int kSelCap = 48 * 1024;

// Order-preserving key: larger score, larger key; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// (kv_len_out may be kv_len: the copies write min(kv_len, keep) there while other
// blocks of theirs read it, which gives both the same number of tokens; the
// selection, which needs kv_len itself, writes it only where there are no copies,
// and every length is 0.)
__device__ __forceinline__ int evict_len(const PagedParams& g, int s) {
    int kv = g.kv_len[s];
    if (!paged_len_ok(kv, g.max_kv)) {
        flag_meta(g.status);
        kv = 0;
    }
    return kv;
}

__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(PagedEvictParams p, int cap) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[kHistCopies][kBins];
    __shared__ uint32_t s_sum[kSelWarps], s_prefix, s_want;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, s = blockIdx.y;
    const int kv = evict_len(p.g, s);
    const int len = min(kv, p.keep), recent = min(p.recent, kv);
    const int64_t row = static_cast<int64_t>(s) * p.g.kv_heads + h;
    const float* sc = p.scores + row * p.score_stride;
    int32_t* kept = p.kept + row * p.keep;
    if (p.g.max_kv == 0 && h == 0 && tid == 0) p.kv_len_out[s] = len;
    for (int i = len + tid; i < p.keep; i += kSelThreads) {
        kept[i] = -1;
        if (p.scores_out) p.scores_out[row * p.keep + i] = 0.f;
    }
    const int cand = kv - recent, want = len - recent;  // candidates, and how many of them stay
    for (int i = (want == cand ? 0 : want) + tid; i < len; i += kSelThreads) {
        kept[i] = i < want ? i : cand + i - want;
    }
    if (want == cand || want == 0) return;

    const bool staged = cand <= cap;
    auto key = [&](int i) { return staged ? keys[i] : score_key(__ldg(sc + i)); };
    // ---- the want-th largest key
    uint32_t prefix = 0, left = want;
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? kShift[0] : pass == 1 ? kShift[1] : kShift[2];
        const int bits = pass == 2 ? kBits[2] : kBits[0];
        for (int i = tid; i < kHistCopies * kBins; i += kSelThreads) hist[i / kBins][i % kBins] = 0;
        __syncthreads();
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + bits);
        auto count = [&](uint32_t k) {
            if ((k & mask) == prefix) atomicAdd(&hist[lane & (kHistCopies - 1)][(k >> shift) & ((1u << bits) - 1u)], 1u);
        };
        if (pass == 0) {
            // the scores, many on their way at a time
            for (int i0 = tid; i0 < cand; i0 += kBatch * kSelThreads) {
                float x[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    x[u] = i0 + u * kSelThreads < cand ? __ldg(sc + i0 + u * kSelThreads) : 0.f;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kSelThreads;
                    if (i >= cand) break;
                    const uint32_t k = score_key(x[u]);
                    if (staged) keys[i] = k;
                    count(k);
                }
            }
        } else {
#pragma unroll 4
            for (int i = tid; i < cand; i += kSelThreads) count(key(i));
        }
        __syncthreads();
        // thread l: bins 2047 - 2 l and 2046 - 2 l, the highest first
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = hist[0][kBins - 1 - 2 * tid - i] + hist[1][kBins - 1 - 2 * tid - i];
        uint32_t above = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
            if (lane >= o) above += v;
        }
        if (lane == 31) s_sum[warp] = above;
        __syncthreads();
        uint32_t before = lane < warp ? s_sum[lane] : 0u;
        before = __reduce_add_sync(0xffffffffu, before);
        above += before - (c[0] + c[1]);  // keys in higher bins
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (above < left && left <= above + c[i]) {
                s_prefix = prefix | (static_cast<uint32_t>(kBins - 1 - 2 * tid - i) << shift);
                s_want = left - above;
            }
            above += c[i];
        }
        __syncthreads();
        prefix = s_prefix;
        left = s_want;
        __syncthreads();
    }
    // keys over `prefix` stay, and the first `left` of those equal to it
    const int seg = (cand + kSelThreads - 1) / kSelThreads * 32;  // scores of a warp
    const int a = min(cand, warp * seg), b = min(cand, a + seg);
    int gt = 0, eq = 0;
#pragma unroll 4
    for (int i = a; i < b; i += 32) {
        const uint32_t k = i + lane < b ? key(i + lane) : 0u;
        const bool in = i + lane < b;
        gt += __popc(__ballot_sync(0xffffffffu, in && k > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, in && k == prefix));
    }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    gt = eq = 0;
    for (int w = 0; w < warp; ++w) {
        gt += s_gt[w];
        eq += s_eq[w];
    }
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
    for (int i = a; i < b; i += 32) {
        const bool in = i + lane < b;
        const uint32_t k = in ? key(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && k > prefix), be = __ballot_sync(0xffffffffu, in && k == prefix);
        const int e = eq + __popc(be & below);
        const bool take = in && (k > prefix || (k == prefix && e < static_cast<int>(left)));
        if (take) {
            const int to = gt + __popc(bg & below) + min(e, static_cast<int>(left));
            kept[to] = i + lane;
        }
        gt += __popc(bg);
        eq += __popc(be);
    }
}

// 64 tokens by 256 threads: 95 us for the batch above; 32 by 128 96, 64 by 128
// 108, 128 by 512 102.
constexpr int kGatherTokens = 64;
constexpr int kGatherThreads = 256;
constexpr int kGatherPieces = 16;  // 16-byte pieces of a V row in shared memory at a time

template <int D>
__global__ void __launch_bounds__(kGatherThreads, 1536 / kGatherThreads) paged_gather_kernel(PagedEvictParams p) {
    constexpr int kRow = 16 * kGatherPieces + 16;  // bytes of a staged row: 16-byte aligned, spread over the banks
    __shared__ int64_t src[kGatherTokens];         // (page, head, place) of each token, -1: none
    __shared__ int64_t dst[kGatherTokens / 16];    // of each 16 tokens' destination
    __shared__ int64_t piece[kGatherTokens];       // (page, head, first place) of each piece
    __shared__ int place[kGatherTokens];           // 16 x piece + byte of each token, -1: none
    __shared__ int s_pieces;
    __shared__ __align__(16) uint8_t in[D * kRow];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, s = blockIdx.z, i0 = blockIdx.x * kGatherTokens;
    const int kv = evict_len(p.g, s);
    const int n = min(kGatherTokens, min(kv, p.keep) - i0);
    if (i0 == 0 && h == 0 && tid == 0) p.kv_len_out[s] = min(kv, p.keep);
    if (n <= 0) return;
    const int shift = p.g.page_shift, P = 1 << shift;
    if (tid < kGatherTokens) {
        int64_t a = -1;
        if (tid < n) {
            const int64_t row = static_cast<int64_t>(s) * p.g.kv_heads + h;
            const int j = __ldg(p.kept + row * p.keep + i0 + tid);
            if (p.scores_out) p.scores_out[row * p.keep + i0 + tid] = __ldg(p.scores + row * p.score_stride + j);
            const int page = load_page(p.g, s, j >> shift);
            if (page >= 0) a = (static_cast<int64_t>(page) * p.g.kv_heads + h) * P + (j & (P - 1));
        }
        src[tid] = a;
        if ((tid & 15) == 0) {
            int64_t b = -1;
            const int i = i0 + tid;
            if (tid < n) {
                const int to = __ldg(p.dst_table + static_cast<int64_t>(s) * p.dst_pages + (i >> shift));
                if (paged_page_ok(to, p.g.pages))
                    b = (static_cast<int64_t>(to) * p.g.kv_heads + h) * P + (i & (P - 1));
                else
                    flag_meta(p.g.status);
            }
            dst[tid >> 4] = b;
        }
    }
    __syncthreads();
    // K rows and scales are on their way while the pieces of V are listed
    constexpr int kPieces = D / 16, kCopies = kGatherTokens * kPieces / kGatherThreads;
    uint4 krow[kCopies];
#pragma unroll
    for (int x = 0; x < kCopies; ++x) {
        const int i = tid + x * kGatherThreads, t = i / kPieces, c = i % kPieces;
        krow[x] = src[t] >= 0 ? ldg_nc_na_v4(p.g.kcodes + src[t] * D + 16 * c) : make_uint4(0, 0, 0, 0);
    }
    const int st = tid - 64;  // the token whose scales this thread copies
    const bool scales = st >= 0 && st < kGatherTokens && src[st] >= 0 && dst[st >> 4] >= 0;
    uint8_t kscale = 0, vscale = 0;
    if (scales) {
        kscale = __ldg(p.g.kscale + src[st]);
        vscale = __ldg(p.g.vscale + src[st]);
    }
    // the 16-byte pieces of V rows that hold the tokens (which ascend: equal
    // pieces are neighbours; a token on a bad page has none)
    if (warp == 0) {
        int count = 0;
#pragma unroll
        for (int k = 0; k < kGatherTokens; k += 32) {
            const int64_t a = src[k + lane], before = k + lane > 0 ? src[k + lane - 1] : -1;
            const bool first = a >= 0 && (before < 0 || (before >> 4) != (a >> 4));
            const uint32_t firsts = __ballot_sync(0xffffffffu, first);
            const int at = count + __popc(firsts & ((2u << lane) - 1u)) - 1;
            if (first) piece[at] = a & ~static_cast<int64_t>(15);
            place[k + lane] = a < 0 ? -1 : 16 * at + static_cast<int>(a & 15);
            count += __popc(firsts);
        }
        if (lane == 0) s_pieces = count;
    }
    __syncthreads();
    // V: element (d, place) of (page, head) b is byte (b D + d) P + place.
    // Thread: tokens 4 w .. 4 w + 3 of some dims.
    constexpr int kWords = kGatherTokens / 4;
    const int pieces = s_pieces, w = tid % kWords;
    const int64_t to = dst[w >> 2];
    for (int first = 0; first < pieces || first == 0; first += kGatherPieces) {
        const int here = min(kGatherPieces, pieces - first);
        // four pieces of a row by neighbouring lanes: they often lie side by side
        for (int k = tid & 3; k < here; k += 4) {
            const int64_t b = piece[first + k];
            const uint8_t* from = p.g.vcodes + (b >> shift) * D * P + (b & (P - 1));
#pragma unroll
            for (int d = tid >> 2; d < D; d += kGatherThreads / 4)
                cp_async16(in + d * kRow + 16 * k, from + (static_cast<uint32_t>(d) << shift));
        }
        if (first == 0) {
#pragma unroll
            for (int x = 0; x < kCopies; ++x) {
                const int i = tid + x * kGatherThreads, t = i / kPieces, c = i % kPieces;
                if (src[t] >= 0 && dst[t >> 4] >= 0)
                    *reinterpret_cast<uint4*>(p.g.kcodes + (dst[t >> 4] + (t & 15)) * D + 16 * c) = krow[x];
            }
            if (scales) {
                p.g.kscale[dst[st >> 4] + (st & 15)] = kscale;
                p.g.vscale[dst[st >> 4] + (st & 15)] = vscale;
            }
        }
        cp_async_wait_all();
        __syncthreads();
        if (to >= 0) {
            int at[4];
            bool have[4], all = true;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int v = place[4 * w + x];
                have[x] = v >= 16 * first && v < 16 * (first + here);
                at[x] = have[x] ? v - 16 * first : 0;
                all &= have[x];
            }
            uint8_t* out = p.g.vcodes + (to >> shift) * D * P + (to & (P - 1)) + 4 * (w & 3);
#pragma unroll 4
            for (int d = tid / kWords; d < D; d += kGatherThreads / kWords) {
                const uint8_t* row = in + d * kRow;
                uint8_t* o = out + (static_cast<uint32_t>(d) << shift);
                if (all) {
                    *reinterpret_cast<uint32_t*>(o) = row[at[0]] | (row[at[1]] << 8) | (row[at[2]] << 16) |
                                                      (static_cast<uint32_t>(row[at[3]]) << 24);
                } else {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (have[x]) o[x] = row[at[x]];
                }
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, int D, cudaStream_t s) {
    static std::atomic<uint64_t> configured{0};
    const int cap = std::min(kSelCap, std::max(1, p.g.max_kv));
    cudaError_t e = smem_limit_once(paged_select_kernel, kSelCap * 4, configured);
    if (e != cudaSuccess) return e;
    paged_select_kernel<<<dim3(p.g.kv_heads, p.g.seqs), kSelThreads, cap * 4, s>>>(p, cap);
    e = cudaGetLastError();
    const int most = std::min(p.keep, p.g.max_kv);
    if (e != cudaSuccess || most == 0) return e;
    const dim3 grid((most + kGatherTokens - 1) / kGatherTokens, p.g.kv_heads, p.g.seqs);
    if (D == 128)
        paged_gather_kernel<128><<<grid, kGatherThreads, 0, s>>>(p);
    else
        paged_gather_kernel<64><<<grid, kGatherThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rc
