// rc_paged4_host.cu -- the C ABI of the rotary forms and of the 4-bit paged cache
// (include/rc.h): argument checks, parameter blocks, launches.
#include <cstring>

#include "rc_nvtx.h"
#include "rc_paged_host.h"

using namespace rc;

namespace {

constexpr double kTwoPi = 6.283185307179586476925;

bool head_dim_ok(int D) { return D >= 8 && D <= RC_ROPE_MAX_HEAD_DIM && D % 8 == 0; }

bool form_ok(const rc_rope_form* f) {
    if (!f || !head_dim_ok(f->head_dim) || f->axes < 1 || f->axes > RC_ROPE_MAX_AXES) return false;
    if (f->first < 0 || f->first % 2 || f->dims < 2 || f->dims % 2 || f->dims > f->head_dim || f->first > f->head_dim - f->dims) return false;
    if (f->layout != RC_ROPE_PAIRS && f->layout != RC_ROPE_HALVES) return false;
    if (!(f->gain >= 0x1p-16f && f->gain <= 16.f)) return false;
    for (int i = 0; i < f->dims / 2; ++i)
        if (f->axis[i] >= f->axes) return false;
    return true;
}

void copy_form(RopeFormDev* d, const rc_rope_form* f) {
    std::memcpy(d->turns, f->turns, sizeof(d->turns));
    std::memcpy(d->axis, f->axis, sizeof(d->axis));
    d->head_dim = f->head_dim;
    d->first = f->first;
    d->dims = f->dims;
    d->layout = f->layout;
    d->gain = f->gain;
}

// Frequency of pair r of w, stretched.
double frequency(const rc_rope_spec& s, int r, int w) {
    double base = s.base;
    if (s.scaling == RC_ROPE_SCALE_BASE && w > 1) base *= std::pow(s.factor, static_cast<double>(w) / (w - 1));
    const double theta = std::pow(base, -static_cast<double>(r) / w);
    if (s.scaling == RC_ROPE_SCALE_LINEAR) return theta / s.factor;
    if (s.scaling == RC_ROPE_SCALE_PARTS) {
        const double keep = std::min(1.0, std::max(0.0, (s.context * theta / kTwoPi - s.low) / (s.high - s.low)));
        return theta * (keep + (1.0 - keep) / s.factor);
    }
    return theta;
}

}  // namespace

extern "C" {

int rc_rope_form_init(rc_rope_form* form, const rc_rope_spec* spec) {
    if (!form || !spec) return RC_ERR_ARG;
    const rc_rope_spec s = *spec;
    if (!head_dim_ok(s.head_dim)) return RC_ERR_UNSUPPORTED;
    if (s.first < 0 || s.first % 2 || s.dims < 2 || s.dims % 2 || s.dims > s.head_dim || s.first > s.head_dim - s.dims) return RC_ERR_ARG;
    if ((s.layout != RC_ROPE_PAIRS && s.layout != RC_ROPE_HALVES) || s.axes < 1 || s.axes > RC_ROPE_MAX_AXES) return RC_ERR_ARG;
    if (!(s.base > 1.0) || !(s.base <= 1e9) || (s.flags & ~RC_ROPE_SHARED_FREQS)) return RC_ERR_ARG;
    if (s.scaling < RC_ROPE_SCALE_NONE || s.scaling > RC_ROPE_SCALE_PARTS) return RC_ERR_ARG;
    if (s.scaling != RC_ROPE_SCALE_NONE && !(s.factor >= 1.0 && s.factor <= 1e6)) return RC_ERR_ARG;
    if (s.scaling == RC_ROPE_SCALE_PARTS &&
        (!(s.context > 0.0 && s.context <= 0x1p31) || !(s.low >= 0.0) || !(s.high > s.low) || !(s.high <= 0x1p31)))
        return RC_ERR_ARG;
    if (!(s.gain >= 0x1p-16f && s.gain <= 16.f)) return RC_ERR_ARG;
    int64_t sum = 0;
    for (int a = 0; a < s.axes; ++a) {
        if (s.sections[a] < 0) return RC_ERR_ARG;
        sum += s.sections[a];
    }
    if (sum != s.dims / 2) return RC_ERR_ARG;
    std::memset(form, 0, sizeof(*form));
    form->head_dim = s.head_dim;
    form->first = s.first;
    form->dims = s.dims;
    form->layout = s.layout;
    form->axes = s.axes;
    form->gain = s.gain;
    int i = 0;
    for (int a = 0; a < s.axes; ++a)
        for (int r = 0; r < s.sections[a]; ++r, ++i) {
            form->turns[i] = turns_of((s.flags & RC_ROPE_SHARED_FREQS) ? frequency(s, i, s.dims / 2) : frequency(s, r, s.sections[a]));
            form->axis[i] = static_cast<uint8_t>(a);
        }
    return RC_OK;
}

int rc_rope_turn(const rc_rope_form* form, const void* x, int64_t x_stride, void* out, int64_t out_stride, int dtype,
                 int64_t n, int heads, const int32_t* positions, int64_t pos_stride, int back, void* stream) {
    const NvtxRange range("rc_rope_turn");
    if ((dtype != RC_BF16 && dtype != RC_F32) || n < 0 || heads < 1 || !form_ok(form)) return RC_ERR_ARG;
    if (n == 0) return RC_OK;
    if (!x || !out || !positions || !aligned16(x) || !aligned16(out)) return RC_ERR_ARG;
    const int unit = dtype == RC_BF16 ? 8 : 4;
    const int64_t row = static_cast<int64_t>(heads) * form->head_dim;
    if (!stride_ok(x_stride, row, unit) || !stride_ok(out_stride, row, unit) || pos_stride < n) return RC_ERR_ARG;
    if (n > 0x7fffffff || row > 0x7fffffff) return RC_ERR_UNSUPPORTED;
    const bool in_place = x == out && x_stride == out_stride;
    if (!in_place && meet({x, x_stride, n, row}, {out, out_stride, n, row}, dtype == RC_BF16 ? 2 : 4)) return RC_ERR_ARG;
    const int st = ready();
    if (st != RC_OK) return st;
    RopeFormParams p{};
    copy_form(&p.form, form);
    p.x = x;
    p.out = out;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.pos_stride = pos_stride;
    p.n = n;
    p.pos = positions;
    p.heads = heads;
    p.back = back;
    return launch_rope_form(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK : RC_ERR_CUDA;
}

int rc_paged4_write(const rc_paged4_view* view, const rc_paged_batch* batch, const void* K_bf16, int64_t k_stride,
                    const void* V_bf16, int64_t v_stride, const int32_t* positions, int64_t pos_stride,
                    const rc_rope_form* form, void* stream) {
    const NvtxRange range("rc_paged4_write");
    Paged4WriteParams p{};
    int st = check_paged(view, batch, true, &p.g);
    if (st != RC_OK) return st;
    if (form && (!form_ok(form) || form->head_dim != view->head_dim)) return RC_ERR_ARG;
    if (p.g.tokens == 0 || p.g.max_new == 0 || p.g.max_kv == 0) return RC_OK;
    if (!K_bf16 || !V_bf16 || (form && !positions) || !aligned16(K_bf16) || !aligned16(V_bf16)) return RC_ERR_ARG;
    const int64_t row = static_cast<int64_t>(view->kv_heads) * view->head_dim;
    if (!stride_ok(k_stride, row, 8) || !stride_ok(v_stride, row, 8) || (form && pos_stride < p.g.tokens)) return RC_ERR_ARG;
    if (paged_write_blocks(p.g) > kMaxBlocks) return RC_ERR_UNSUPPORTED;
    st = ready();
    if (st != RC_OK) return st;
    p.form.gain = 1.f;
    if (form) copy_form(&p.form, form);
    p.K = static_cast<const __nv_bfloat16*>(K_bf16);
    p.V = static_cast<const __nv_bfloat16*>(V_bf16);
    p.pos = positions;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pos_stride = pos_stride;
    return launch_paged4_write(p, view->head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess ? RC_OK : RC_ERR_CUDA;
}

int rc_paged4_attend(const rc_paged4_view* view, const rc_paged_batch* batch, const void* Q_bf16, int64_t q_stride,
                     int heads, void* out_bf16, int64_t out_stride, float* lse, int causal, void* stream) {
    const NvtxRange range("rc_paged4_attend");
    PagedAttnParams p{};
    int st = check_attend(view, batch, Q_bf16, q_stride, heads, out_bf16, out_stride, lse, causal, &p);
    if (st != RC_OK || p.q == nullptr) return st;
    return launch_paged4_attention(p, view->head_dim, kPartFloats, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? RC_OK
               : RC_ERR_CUDA;
}

int rc_paged4_status(const rc_paged4_view* view, void* stream) {
    return view ? paged_status(view->workspace, static_cast<cudaStream_t>(stream)) : RC_ERR_ARG;
}

}  // extern "C"
