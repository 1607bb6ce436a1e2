// rc_paged_host.cu -- the C ABI of the several-axes rotary positions and the
// paged cache (include/rc.h): argument checks, parameter blocks, launches.
#include <cstring>

#include "rc_nvtx.h"
#include "rc_paged_host.h"

using namespace rc;

namespace {

bool plan_ok(const rc_rope_plan* plan, int D) {
    if (!plan || plan->head_dim != D || plan->axes < 1 || plan->axes > RC_ROPE_MAX_AXES) return false;
    for (int i = 0; i < D / 2; ++i)
        if (plan->axis[i] >= plan->axes) return false;
    return true;
}

void copy_plan(RopePlanDev* d, const rc_rope_plan* plan) {
    std::memcpy(d->turns, plan->turns, sizeof(d->turns));
    std::memcpy(d->axis, plan->axis, sizeof(d->axis));
}

}  // namespace

extern "C" {

int rc_rope_plan_init(rc_rope_plan* plan, int head_dim, int axes, const int* sections, double base, unsigned flags) {
    if (!plan || !sections) return RC_ERR_ARG;
    if (head_dim != 64 && head_dim != 128) return RC_ERR_UNSUPPORTED;
    if (axes < 1 || axes > RC_ROPE_MAX_AXES || !(base > 1.0) || !(base <= 1e9) || (flags & ~RC_ROPE_SHARED_FREQS))
        return RC_ERR_ARG;
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0) return RC_ERR_ARG;
        sum += sections[a];
    }
    if (sum != head_dim / 2) return RC_ERR_ARG;
    std::memset(plan, 0, sizeof(*plan));
    plan->head_dim = head_dim;
    plan->axes = axes;
    int i = 0;
    for (int a = 0; a < axes; ++a)
        for (int r = 0; r < sections[a]; ++r, ++i) {
            const double theta = (flags & RC_ROPE_SHARED_FREQS) ? std::pow(base, -2.0 * i / head_dim)
                                                                : std::pow(base, -static_cast<double>(r) / sections[a]);
            plan->turns[i] = turns_of(theta);
            plan->axis[i] = static_cast<uint8_t>(a);
        }
    return RC_OK;
}

int rc_rope_axes(const rc_rope_plan* plan, const void* x, int64_t x_stride, void* out, int64_t out_stride, int dtype,
                 int64_t n, int heads, const int32_t* positions, int64_t pos_stride, int inverse, void* stream) {
    const NvtxRange range("rc_rope_axes");
    if (!plan || (dtype != RC_BF16 && dtype != RC_F32) || n < 0 || heads < 1) return RC_ERR_ARG;
    if (plan->head_dim != 64 && plan->head_dim != 128) return RC_ERR_ARG;
    if (!plan_ok(plan, plan->head_dim)) return RC_ERR_ARG;
    if (n == 0) return RC_OK;
    if (!x || !out || !positions || !aligned16(x) || !aligned16(out)) return RC_ERR_ARG;
    const int unit = dtype == RC_BF16 ? 8 : 4;
    const int64_t row = static_cast<int64_t>(heads) * plan->head_dim;
    if (!stride_ok(x_stride, row, unit) || !stride_ok(out_stride, row, unit) || pos_stride < n) return RC_ERR_ARG;
    if (n > 0x7fffffff || row > 0x7fffffff) return RC_ERR_UNSUPPORTED;
    if (!(x == out && x_stride == out_stride) &&
        meet({x, x_stride, n, row}, {out, out_stride, n, row}, dtype == RC_BF16 ? 2 : 4))
        return RC_ERR_ARG;
    const int st = ready();
    if (st != RC_OK) return st;
    RopeAxesParams p{};
    copy_plan(&p.rope, plan);
    p.x = x;
    p.out = out;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.pos_stride = pos_stride;
    p.n = n;
    p.pos = positions;
    p.heads = heads;
    p.inverse = inverse;
    return launch_rope_axes(p, plan->head_dim, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK
                                                                                                        : RC_ERR_CUDA;
}

int rc_paged_write(const rc_paged_view* view, const rc_paged_batch* batch, const void* K_bf16, int64_t k_stride,
                   const void* V_bf16, int64_t v_stride, const int32_t* positions, int64_t pos_stride,
                   const rc_rope_plan* plan, void* stream) {
    const NvtxRange range("rc_paged_write");
    PagedWriteParams p{};
    int st = check_paged(view, batch, true, &p.g);
    if (st != RC_OK) return st;
    if (!plan_ok(plan, view->head_dim)) return RC_ERR_ARG;
    if (p.g.tokens == 0 || p.g.max_new == 0 || p.g.max_kv == 0) return RC_OK;
    if (!K_bf16 || !V_bf16 || !positions || !aligned16(K_bf16) || !aligned16(V_bf16)) return RC_ERR_ARG;
    const int64_t row = static_cast<int64_t>(view->kv_heads) * view->head_dim;
    if (!stride_ok(k_stride, row, 8) || !stride_ok(v_stride, row, 8) || pos_stride < p.g.tokens) return RC_ERR_ARG;
    if (paged_write_blocks(p.g) > kMaxBlocks) return RC_ERR_UNSUPPORTED;
    st = ready();
    if (st != RC_OK) return st;
    copy_plan(&p.rope, plan);
    p.K = static_cast<const __nv_bfloat16*>(K_bf16);
    p.V = static_cast<const __nv_bfloat16*>(V_bf16);
    p.pos = positions;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pos_stride = pos_stride;
    return launch_paged_write(p, view->head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK : RC_ERR_CUDA;
}

int rc_paged_attend(const rc_paged_view* view, const rc_paged_batch* batch, const void* Q_bf16, int64_t q_stride,
                    int heads, void* out_bf16, int64_t out_stride, float* lse, int causal, void* stream) {
    const NvtxRange range("rc_paged_attend");
    PagedAttnParams p{};
    int st = check_attend(view, batch, Q_bf16, q_stride, heads, out_bf16, out_stride, lse, causal, &p);
    if (st != RC_OK || p.q == nullptr) return st;
    return launch_paged_attention(p, view->head_dim, kPartFloats, kCounters, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? RC_OK
               : RC_ERR_CUDA;
}

int rc_paged_accumulate(const rc_paged_view* view, const rc_paged_batch* batch, const void* Q_bf16, int64_t q_stride,
                        int heads, const float* lse, const float* scores, float* out, int64_t score_stride, int causal,
                        void* stream) {
    const NvtxRange range("rc_paged_accumulate");
    PagedScoreParams p{};
    int st = check_paged(view, batch, true, &p.g);
    if (st != RC_OK) return st;
    if (heads < 1 || heads > 65535 || heads % view->kv_heads != 0 || score_stride < p.g.max_kv) return RC_ERR_ARG;
    if (p.g.max_kv == 0) return RC_OK;
    if (!scores || !out) return RC_ERR_ARG;
    const int64_t lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    if (scores != out && meet({scores, score_stride, lists, p.g.max_kv}, {out, score_stride, lists, p.g.max_kv}, 4))
        return RC_ERR_ARG;
    if (p.g.tokens > 0 && (!Q_bf16 || !lse || !aligned16(Q_bf16))) return RC_ERR_ARG;
    if (p.g.tokens > 0 && !stride_ok(q_stride, static_cast<int64_t>(heads) * view->head_dim, 8)) return RC_ERR_ARG;
    if (static_cast<int64_t>(p.g.max_new) * (heads / view->kv_heads) > (1 << 30)) return RC_ERR_UNSUPPORTED;
    st = ready();
    if (st != RC_OK) return st;
    p.q = static_cast<const __nv_bfloat16*>(Q_bf16);
    p.q_stride = q_stride;
    p.lse = lse;
    p.scores = scores;
    p.out = out;
    p.score_stride = score_stride;
    p.heads = heads;
    p.group = heads / view->kv_heads;
    p.causal = causal;
    p.sm_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(view->head_dim)));
    p.wait_ns = g_paged_wait_ns.load(std::memory_order_relaxed);
    return launch_paged_scores(p, view->head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK
                                                                                                    : RC_ERR_CUDA;
}

int rc_paged_evict(const rc_paged_view* view, const rc_paged_batch* batch, const float* scores, int64_t score_stride,
                   int keep, int recent, const int32_t* dst_table, int dst_pages, int32_t* kept, int32_t* kv_len_out,
                   float* scores_out, void* stream) {
    const NvtxRange range("rc_paged_evict");
    PagedEvictParams p{};
    int st = check_paged(view, batch, false, &p.g);
    if (st != RC_OK) return st;
    if (keep < 1 || recent < 0 || recent > keep || dst_pages < 0) return RC_ERR_ARG;
    if (!kept || !kv_len_out || score_stride < p.g.max_kv) return RC_ERR_ARG;
    const int most = keep < p.g.max_kv ? keep : p.g.max_kv;
    if (static_cast<int64_t>(dst_pages) * view->page_tokens < most) return RC_ERR_ARG;
    if (most > 0 && (!scores || !dst_table)) return RC_ERR_ARG;
    if (keep > (1 << 24)) return RC_ERR_UNSUPPORTED;
    const int64_t lists = static_cast<int64_t>(p.g.seqs) * p.g.kv_heads;
    if (scores_out && meet({scores, score_stride, lists, p.g.max_kv}, {scores_out, lists * keep, 1, lists * keep}, 4))
        return RC_ERR_ARG;
    st = ready();
    if (st != RC_OK) return st;
    p.scores = scores;
    p.score_stride = score_stride;
    p.keep = keep;
    p.recent = recent;
    p.dst_pages = dst_pages;
    p.dst_table = dst_table;
    p.kept = kept;
    p.kv_len_out = kv_len_out;
    p.scores_out = scores_out;
    return launch_paged_evict(p, view->head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK : RC_ERR_CUDA;
}

int rc_paged_status(const rc_paged_view* view, void* stream) {
    return view ? paged_status(view->workspace, static_cast<cudaStream_t>(stream)) : RC_ERR_ARG;
}

int rc_paged_set_wait_limit(uint64_t ns) {
    if (ns > 60000000000ull) return RC_ERR_ARG;
    g_paged_wait_ns.store(ns, std::memory_order_relaxed);
    return RC_OK;
}

}  // extern "C"
