// rc_paged_evict.cu -- cutting sequences to a budget by accumulated attention
// weight.
//
// paged_select_kernel: one block per (sequence, KV head) finds the budget's
//    threshold among the scores by radix selection, 8 bits of the ordered key a
//    pass (the keys stay in shared memory while they fit), then lists the kept
//    indices in ascending order: each warp counts in its own run of scores with
//    ballots, the counts are summed over the warps, and each warp writes its
//    run.  Ties at the threshold go to the lowest index.
// paged_gather_kernel: copies the kept tokens to the new pages: bound by
//    memory.  K rows go 16 bytes a thread; a V row's codes (one per token) go
//    a byte a lane, 32 kept tokens side by side, so that the loads of a warp
//    fall into few sectors and its stores into one.
#include <algorithm>

#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHistCopies = 8;           // histograms a lane group has to itself: neighbours often share a bin
constexpr int kSelCap = 48 * 1024;       // keys kept in shared memory

// Order-preserving key: larger score, larger key; -0 as +0, NaN above all.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int evict_len(const PagedParams& g, int s) {
    int kv = __ldg(g.kv_len + s);
    if (kv < 0 || kv > g.max_kv) {
        flag_meta(g.status);
        kv = 0;
    }
    return kv;
}

__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(PagedEvictParams p, int cap) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[kHistCopies][256];
    __shared__ uint32_t s_prefix, s_want;
    __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, s = blockIdx.y;
    const int kv = evict_len(p.g, s);
    const int len = min(kv, p.keep), recent = min(p.recent, kv);
    const int64_t row = static_cast<int64_t>(s) * p.g.kv_heads + h;
    const float* sc = p.scores + row * p.score_stride;
    int32_t* kept = p.kept + row * p.keep;
    float* sout = p.scores_out ? p.scores_out + row * p.keep : nullptr;
    if (h == 0 && tid == 0) p.kv_len_out[s] = len;
    for (int i = len + tid; i < p.keep; i += kSelThreads) {
        kept[i] = -1;
        if (sout) sout[i] = 0.f;
    }
    const int cand = kv - recent, want = len - recent;  // candidates, and how many of them stay
    for (int i = (want == cand ? 0 : want) + tid; i < len; i += kSelThreads) {
        const int j = i < want ? i : cand + i - want;
        kept[i] = j;
        if (sout) sout[i] = sc[j];
    }
    if (want == cand || want == 0) return;

    const bool staged = cand <= cap;
    if (staged)
        for (int i = tid; i < cand; i += kSelThreads) keys[i] = score_key(__ldg(sc + i));
    auto key = [&](int i) { return staged ? keys[i] : score_key(__ldg(sc + i)); };
    // ---- the want-th largest key
    uint32_t prefix = 0, left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < kHistCopies * 256; i += kSelThreads) hist[i >> 8][i & 255] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int i = tid; i < cand; i += kSelThreads) {
            const uint32_t k = key(i);
            if ((k & mask) == prefix) atomicAdd(&hist[lane & (kHistCopies - 1)][(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l: bins 255 - 8 l down to 248 - 8 l
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = 0;
                for (int k = 0; k < kHistCopies; ++k) c[i] += hist[k][255 - 8 * lane - i];
                sum += c[i];
            }
            uint32_t above = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += v;
            }
            above -= sum;  // keys in higher bins
            if (above < left && left <= above + sum) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < left && left <= above + c[i]) {
                        s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
                        s_want = left - above;
                    }
                    above += c[i];
                }
            }
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
    for (int i = a; i < b; i += 32) {
        const bool in = i + lane < b;
        const uint32_t k = in ? key(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, in && k > prefix), be = __ballot_sync(0xffffffffu, in && k == prefix);
        const int e = eq + __popc(be & below);
        const bool take = in && (k > prefix || (k == prefix && e < static_cast<int>(left)));
        if (take) {
            const int to = gt + __popc(bg & below) + min(e, static_cast<int>(left));
            kept[to] = i + lane;
            if (sout) sout[to] = __ldg(sc + i + lane);
        }
        gt += __popc(bg);
        eq += __popc(be);
    }
}

constexpr int kGatherTokens = 64;
constexpr int kGatherThreads = 256;

template <int D>
__global__ void __launch_bounds__(kGatherThreads) paged_gather_kernel(PagedEvictParams p) {
    __shared__ int64_t src[kGatherTokens];  // row (page, head, place) of each token, -1: none
    __shared__ int64_t dst[kGatherTokens];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y, s = blockIdx.z, i0 = blockIdx.x * kGatherTokens;
    const int kv = evict_len(p.g, s);
    const int n = min(kGatherTokens, min(kv, p.keep) - i0);
    if (n <= 0) return;
    const int shift = p.g.page_shift, P = 1 << shift;
    if (tid < kGatherTokens) {
        int64_t a = -1, b = -1;
        if (tid < n) {
            const int64_t row = static_cast<int64_t>(s) * p.g.kv_heads + h;
            const int j = __ldg(p.kept + row * p.keep + i0 + tid), i = i0 + tid;
            const int page = load_page(p.g, s, j >> shift);
            int to = __ldg(p.dst_table + static_cast<int64_t>(s) * p.dst_pages + (i >> shift));
            if (to < 0 || to >= p.g.pages) {
                flag_meta(p.g.status);
                to = -1;
            }
            if (page >= 0 && to >= 0) {
                a = (static_cast<int64_t>(page) * p.g.kv_heads + h) * P + (j & (P - 1));
                b = (static_cast<int64_t>(to) * p.g.kv_heads + h) * P + (i & (P - 1));
            }
        }
        src[tid] = a;
        dst[tid] = b;
        if (a >= 0) {
            p.g.kscale[b] = p.g.kscale[a];
            p.g.vscale[b] = p.g.vscale[a];
        }
    }
    __syncthreads();
    constexpr int kPieces = D / 16;
    for (int i = tid; i < n * kPieces; i += kGatherThreads) {
        const int t = i / kPieces, c = i % kPieces;
        if (src[t] >= 0)
            *reinterpret_cast<uint4*>(p.g.kcodes + dst[t] * D + 16 * c) =
                *reinterpret_cast<const uint4*>(p.g.kcodes + src[t] * D + 16 * c);
    }
    // V: element (d, place) of page block `b` is byte (b D + d) P + place
#pragma unroll
    for (int k = 0; k < kGatherTokens / 32; ++k) {
        const int64_t a = src[32 * k + lane], b = dst[32 * k + lane];
        if (a < 0) continue;
        const uint8_t* from = p.g.vcodes + (a >> shift) * D * P + (a & (P - 1));
        uint8_t* to = p.g.vcodes + (b >> shift) * D * P + (b & (P - 1));
        constexpr int kWarps = kGatherThreads / 32;
#pragma unroll 8
        for (int d = warp; d < D; d += kWarps) to[static_cast<int64_t>(d) * P] = from[static_cast<int64_t>(d) * P];
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
