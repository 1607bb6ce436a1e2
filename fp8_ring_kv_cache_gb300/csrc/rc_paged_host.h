// rc_paged_host.h -- what the entry points of the paged caches and of the rotary
// positions share on the host: argument checks, the device check, frequencies.
#pragma once
#include <algorithm>
#include <atomic>
#include <cmath>

#include "rc_paged.cuh"

namespace rc {

constexpr size_t kStatusBytes = 256;
constexpr int kCounters = 16384;
constexpr int64_t kMaxBlocks = 0x7fffffff;  // of a grid's x
constexpr size_t kPartOff = kStatusBytes + sizeof(int) * kCounters;
constexpr size_t kPartFloats = (RC_PAGED_WORKSPACE_BYTES - kPartOff) / sizeof(float);

// The longest one wait of a paged call may take (rc_paged_set_wait_limit).
inline std::atomic<uint64_t> g_paged_wait_ns{2000000000ull};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// RC_OK if the current device is one these kernels are built for.  The answer
// is kept per device index (below 64).
inline int device_ok() {
    static std::atomic<uint64_t> good{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RC_ERR_CUDA;
    const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
    if (good.load(std::memory_order_acquire) & bit) return RC_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return RC_ERR_CUDA;
    if (major != 10 || minor != 3) return RC_ERR_UNSUPPORTED;
    good.fetch_or(bit, std::memory_order_release);
    return RC_OK;
}

// After the argument checks, before the first launch of a call.
inline int ready() {
    if (launch_fault()) return RC_ERR_CUDA;
    if (cudaPeekAtLastError() != cudaSuccess) return RC_ERR_CUDA;
    return device_ok();
}

// theta / 2 pi * 2^64, rounded, for theta in (2^-50, 1] radians: integers, so that
// every machine gives the same (theta is m 2^(e - 53) with a 53-bit m; 2^76 / 2 pi
// has 74 bits).
inline uint64_t turns_of(double theta) {
    constexpr unsigned __int128 kInv = (static_cast<unsigned __int128>(0x28be60db9391054aull) << 12) | 0x7f1u;
    int e = 0;
    const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(theta, &e), 53));
    const int shift = 53 - e + 12;  // 64 .. 115
    return static_cast<uint64_t>((m * kInv + (static_cast<unsigned __int128>(1) << (shift - 1))) >> shift);
}

// Whether two sets of rows share memory: rows of `width` elements of `size` bytes, `stride` elements apart.
struct Rows {
    const void* at;
    int64_t stride, rows, width;
};
inline bool meet(const Rows& x, const Rows& y, int size) {
    if (x.rows < 1 || x.width < 1 || y.rows < 1 || y.width < 1) return false;
    constexpr int64_t kFar = INT64_C(1) << 56;  // rows farther apart than any address (times `size` stays in 64 bits)
    return paged_rows_meet(reinterpret_cast<uintptr_t>(x.at), std::min(x.stride, kFar) * size, x.rows, x.width * size,
                           reinterpret_cast<uintptr_t>(y.at), std::min(y.stride, kFar) * size, y.rows, y.width * size);
}

inline bool stride_ok(int64_t stride, int64_t row, int unit) { return stride >= row && stride % unit == 0; }

// The pool's and the batch's host fields and pointers; fills g.  View: rc_paged_view or rc_paged4_view, whose fields
// have the same names.
template <typename View>
int check_paged(const View* v, const rc_paged_batch* b, bool queries, PagedParams* g) {
    if (!v || !b) return RC_ERR_ARG;
    if (v->head_dim != 64 && v->head_dim != 128) return RC_ERR_UNSUPPORTED;
    int shift = 4;
    while (shift < 8 && (1 << shift) != v->page_tokens) ++shift;
    if (shift == 8) return RC_ERR_UNSUPPORTED;
    if (!v->kcodes || !v->vcodes || !v->kscale || !v->vscale || !v->workspace) return RC_ERR_ARG;
    if (!aligned16(v->kcodes) || !aligned16(v->vcodes) || !aligned16(v->kscale) || !aligned16(v->vscale) ||
        (reinterpret_cast<uintptr_t>(v->workspace) & 255u))
        return RC_ERR_ARG;
    if (v->pages < 1 || v->kv_heads < 1 || v->kv_heads > 1024) return RC_ERR_ARG;
    // blocks of 16 tokens are counted in 32 bits (2^32 of them would be 4 TB of codes at head_dim 64)
    if ((static_cast<int64_t>(v->pages) * v->kv_heads << (shift - 4)) > INT64_C(0xffffffff)) return RC_ERR_UNSUPPORTED;
    if (b->seqs < 1 || b->seqs > 65535 || b->table_pages < 0 || b->tokens < 0 || b->max_new < 0 || b->max_kv < 0)
        return RC_ERR_ARG;
    if (b->max_kv > (1 << 24) || b->max_kv > static_cast<int64_t>(b->table_pages) * v->page_tokens) return RC_ERR_ARG;
    if (!b->kv_len || (b->max_kv > 0 && !b->page_table) || (queries && !b->q_start)) return RC_ERR_ARG;
    g->kcodes = v->kcodes;
    g->vcodes = v->vcodes;
    g->kscale = v->kscale;
    g->vscale = v->vscale;
    g->page_table = b->page_table;
    g->kv_len = b->kv_len;
    g->q_start = b->q_start;
    g->status = static_cast<int*>(v->workspace);
    g->pages = v->pages;
    g->kv_heads = v->kv_heads;
    g->page_shift = shift;
    g->seqs = b->seqs;
    g->table_pages = b->table_pages;
    g->tokens = b->tokens;
    g->max_new = b->max_new < b->tokens ? b->max_new : b->tokens;
    g->max_kv = b->max_kv;
    return RC_OK;
}

// The arguments of an attention over either cache; fills p.  RC_OK with p->q null: there is nothing to do.
template <typename View>
int check_attend(const View* view, const rc_paged_batch* batch, const void* Q_bf16, int64_t q_stride, int heads,
                 void* out_bf16, int64_t out_stride, float* lse, int causal, PagedAttnParams* p) {
    int st = check_paged(view, batch, true, &p->g);
    if (st != RC_OK) return st;
    if (heads < 1 || heads > 65535 || heads % view->kv_heads != 0) return RC_ERR_ARG;
    if (p->g.tokens == 0 || p->g.max_new == 0) return RC_OK;
    if (!Q_bf16 || !out_bf16 || !aligned16(Q_bf16) || !aligned16(out_bf16)) return RC_ERR_ARG;
    const int64_t row = static_cast<int64_t>(heads) * view->head_dim;
    if (!stride_ok(q_stride, row, 8) || !stride_ok(out_stride, row, 8)) return RC_ERR_ARG;
    if (meet({Q_bf16, q_stride, p->g.tokens, row}, {out_bf16, out_stride, p->g.tokens, row}, 2)) return RC_ERR_ARG;
    const int64_t rows_of_head = static_cast<int64_t>(p->g.max_new) * (heads / view->kv_heads);
    if (rows_of_head > (1 << 30) || paged_attend_blocks(p->g, rows_of_head) > kMaxBlocks) return RC_ERR_UNSUPPORTED;
    st = ready();
    if (st != RC_OK) return st;
    p->q = static_cast<const __nv_bfloat16*>(Q_bf16);
    p->q_stride = q_stride;
    p->out = static_cast<__nv_bfloat16*>(out_bf16);
    p->out_stride = out_stride;
    p->lse = lse;
    p->heads = heads;
    p->group = heads / view->kv_heads;
    p->causal = causal;
    p->sm_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(view->head_dim)));
    char* ws = static_cast<char*>(view->workspace);
    p->counters = reinterpret_cast<int*>(ws + kStatusBytes);
    p->part = reinterpret_cast<float*>(ws + kPartOff);
    p->wait_ns = g_paged_wait_ns.load(std::memory_order_relaxed);
    return RC_OK;
}

// Wait for the stream and report what the calls on a workspace found.
inline int paged_status(void* workspace, cudaStream_t s) {
    if (!workspace) return RC_ERR_ARG;
    int st = 0;
    if (cudaMemcpyAsync(&st, workspace, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return RC_ERR_CUDA;
    if (st == 0) return RC_OK;
    if (cudaMemsetAsync(workspace, 0, sizeof(int), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return RC_ERR_CUDA;
    return st == kDevBadMeta ? RC_ERR_ARG : RC_ERR_TIMEOUT;
}

}  // namespace rc
