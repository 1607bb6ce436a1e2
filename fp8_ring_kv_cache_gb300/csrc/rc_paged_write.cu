// rc_paged_write.cu -- new tokens into the pages of their sequences: K turned
// at its positions, then K and V each quantised to E4M3 with one power-of-two
// scale per token and head.
//
// Bound by memory: bf16 K and V are read once, codes and scales written once.
// A block takes 16 cached tokens that lie side by side in a page (an aligned
// run, so that a V row's 16 bytes go out in one store) and walks over some
// heads.  A token's row is held by D / 8 lanes with 16 bytes each, whose
// (cos, sin) do not depend on the head: they are computed once.  V goes
// through shared memory to be transposed.  Tokens of the run that are older
// than the call keep their bytes: a run that is not all new stores the new
// tokens byte by byte.
// The codes and scales of K are those of the exact turn (to 2^-25 (|a| + |b|), what
// cos and sin leave): where the fp32 sum is too close to the middle between two codes,
// or the row's largest to the border between two scales, it is taken again with twice
// the bits.  757
// tokens x 48 heads x 128: 15.9 us (28 MB, 4.1 us at the copy rate; with codes of
// the fp32 sums, some five of which in 4.6 million then are the neighbour's,
// 13.0 us).  What it spends its time on is the issue of the conversions and the
// load of K, V and the positions at the start of each block.
#include "rc_paged.cuh"
#include "rc_turn_pair.cuh"

namespace rc {

namespace {

constexpr int kRun = kWriteRun;

// Exponent of the row's scale and its byte, from the largest magnitude as bits:
// infinities and NaNs are above every number.  open: whether that is within 8 units of
// its last place of a border between two scales, 1.75 x 2^k.
template <int LANES>
__device__ __forceinline__ uint32_t scale_byte(const float (&x)[8], float& inv, bool& bad, bool* open = nullptr) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    bad = top >= 0x7f800000u;
    if (open) *open |= (top << 9) - ((0x600000u - 8u) << 9) <= 16u << 9;  // (the 23 bits of the fraction)
    const int e = scale_exponent(__uint_as_float(top));
    inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e in -124 .. 7: exact
    return bad ? 255u : static_cast<uint32_t>(e + 127);
}

// K's rows of heads h0 .. h1 - 1 of a warp's tokens written again, all from the exact
// sums, where the fp32 sums leave the scale of one of them open.  (Out of line, with the
// angles taken again: what some rows of a million need costs the others little.)
template <int D>
__device__ __noinline__ void write_exact_rows(const PagedWriteParams& p, bool live, int h0, int h1, int c, int row, int page, int place) {
    TurnPair cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        cs[i] = turn_cos_sin_pair(__ldg(p.pos + p.rope.axis[4 * c + i] * p.pos_stride + row), p.rope.turns[4 * c + i]);
    for (int h = h0; h < h1; ++h) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p.K + row * p.k_stride + static_cast<size_t>(h) * D + c * 8));
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(in[i] << 16), b = __uint_as_float(in[i] & 0xFFFF0000u);
            const float2 ch = cs[i].hi, cl = cs[i].lo;
            if (a == 0.f && b == 0.f) {  // (a pair of zeros keeps its sign)
                rotate_pair(a, b, ch.x, ch.y, y[2 * i], y[2 * i + 1]);
            } else {
                y[2 * i] = sum_exactly(a, ch.x, cl.x, -b, ch.y, cl.y);
                y[2 * i + 1] = sum_exactly(a, ch.y, cl.y, b, ch.x, cl.x);
            }
        }
        float inv;
        bool bad;
        const uint32_t kb = scale_byte<D / 8>(y, inv, bad);
        if (!live) continue;
        uint32_t kc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kc[i] = bad ? 0u : e4m3x2(y[2 * i] * inv, y[2 * i + 1] * inv);
        const size_t at = ((static_cast<size_t>(page) * p.g.kv_heads + h) << p.g.page_shift) + place;
        *reinterpret_cast<uint2*>(p.g.kcodes + at * D + c * 8) = make_uint2(kc[0] | (kc[1] << 16), kc[2] | (kc[3] << 16));
        if (c == 0) p.g.kscale[at] = static_cast<uint8_t>(kb);
    }
}

template <int D>
__global__ void __launch_bounds__(kRun * D / 8, 512 / D) paged_write_kernel(const __grid_constant__ PagedWriteParams p, int runs, int heads_per_block) {
    constexpr int LANES = D / 8;  // of one token
    constexpr int kThreads = kRun * LANES;
    constexpr int kRow = D + 16;  // a token's staged codes: 16-byte aligned, rows spread over the banks
    __shared__ __align__(16) uint8_t stage[2][kRun * kRow];
    const int s = blockIdx.x / runs, run = blockIdx.x % runs;
    const Seq q = load_seq(p.g, s);
    if (q.n == 0) return;
    if (q.n > q.kv) {  // new tokens that the length does not count
        if (threadIdx.x == 0) flag_meta(p.g.status);
        return;
    }
    const int first = q.kv - q.n;             // index of the first new token
    const int base = (first & ~(kRun - 1)) + run * kRun;  // index of the run's first token
    if (base >= q.kv) return;
    const int page = load_page(p.g, s, base >> p.g.page_shift);
    if (page < 0) return;
    const int P = 1 << p.g.page_shift, off = base & (P - 1);
    const int tok = threadIdx.x / LANES, c = threadIdx.x % LANES;
    const int index = base + tok;
    const bool live = index >= first && index < q.kv;
    const bool whole = base >= first && base + kRun <= q.kv;
    const int row = q.q0 + (live ? index - first : 0);

    TurnPair cs[4];
    const uint64_t* turns = param_address(p.rope.turns) + 4 * c;
    const uint32_t axes = *reinterpret_cast<const uint32_t*>(param_address(p.rope.axis) + 4 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        cs[i] = turn_cos_sin_pair(__ldg(p.pos + ((axes >> (8 * i)) & 0xffu) * p.pos_stride + row), turns[i]);
    const __nv_bfloat16* kr = p.K + row * p.k_stride + c * 8;
    const __nv_bfloat16* vr = p.V + row * p.v_stride + c * 8;
    const int h0 = blockIdx.y * heads_per_block, h1 = min(p.g.kv_heads, h0 + heads_per_block);
    uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
    if (live) {
        kw = ldg_nc_na_v4(kr + static_cast<size_t>(h0) * D);
        vw = ldg_nc_na_v4(vr + static_cast<size_t>(h0) * D);
    }
    bool open = false;  // a scale of K is
    for (int h = h0; h < h1; ++h) {
        float k[8], v[8], reach[4];
        const uint32_t ki[4] = {kw.x, kw.y, kw.z, kw.w}, vi[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair(__uint_as_float(ki[i] << 16), __uint_as_float(ki[i] & 0xFFFF0000u), cs[i].hi.x, cs[i].hi.y, k[2 * i],
                        k[2 * i + 1]);
            reach[i] = fabsf(__uint_as_float(ki[i] << 16)) + fabsf(__uint_as_float(ki[i] & 0xFFFF0000u));
            v[2 * i] = __uint_as_float(vi[i] << 16);
            v[2 * i + 1] = __uint_as_float(vi[i] & 0xFFFF0000u);
        }
        if (live && h + 1 < h1) {  // the next head is on its way
            kw = ldg_nc_na_v4(kr + static_cast<size_t>(h + 1) * D);
            vw = ldg_nc_na_v4(vr + static_cast<size_t>(h + 1) * D);
        }
        uint32_t kc[4], vc[4];  // pairs of codes
        float inv;
        bool bad;
        // The fp32 sums are within 2^-22 (|a| + |b|) of the exact ones, and |a| + |b| is at
        // most twice the larger of the turned pair: the row's largest magnitude is within
        // 2^-21 of itself, 7 units of the last place at a border between two scales.
        const uint32_t kb = scale_byte<LANES>(k, inv, bad, &open);
        // The fp32 sum is within 2^-22 (|a| + |b|) of the exact one (cos and sin half
        // an ulp each, 2^-25, and three roundings of 2^-24: 2.1e-7).  Where both ends
        // of that range have one code it is the exact sum's; the few others (one
        // pair of 50,000) are summed again.  (A pair of zeros keeps its sign.)
        uint32_t unsure = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float tol = reach[i] * (inv * 0x1p-22f);
            kc[i] = e4m3x2(fmaf(k[2 * i], inv, -tol), fmaf(k[2 * i + 1], inv, -tol));
            if (kc[i] != e4m3x2(fmaf(k[2 * i], inv, tol), fmaf(k[2 * i + 1], inv, tol)) && tol > 0.f) unsure |= 1u << i;
        }
        if (bad) {
#pragma unroll
            for (int i = 0; i < 4; ++i) kc[i] = 0u;
        } else if (unsure) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!(unsure & (1u << i))) continue;
                const float a = __uint_as_float(ki[i] << 16), b = __uint_as_float(ki[i] & 0xFFFF0000u);
                const float2 ch = cs[i].hi, cl = cs[i].lo;
                kc[i] = e4m3x2(sum_exactly(a, ch.x, cl.x, -b, ch.y, cl.y) * inv, sum_exactly(a, ch.y, cl.y, b, ch.x, cl.x) * inv);
            }
        }
        const uint32_t vb = scale_byte<LANES>(v, inv, bad);
#pragma unroll
        for (int i = 0; i < 4; ++i) vc[i] = bad ? 0u : e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
        const size_t ph = static_cast<size_t>(page) * p.g.kv_heads + h;
        uint8_t* st = stage[(h - h0) & 1];
        if (live) {
            *reinterpret_cast<uint2*>(p.g.kcodes + (ph * P + off + tok) * D + c * 8) = make_uint2(kc[0] | (kc[1] << 16), kc[2] | (kc[3] << 16));
            *reinterpret_cast<uint2*>(st + tok * kRow + c * 8) = make_uint2(vc[0] | (vc[1] << 16), vc[2] | (vc[3] << 16));
            if (c == 0) {
                p.g.kscale[ph * P + off + tok] = static_cast<uint8_t>(kb);
                p.g.vscale[ph * P + off + tok] = static_cast<uint8_t>(vb);
            }
        }
        __syncthreads();  // (the other buffer is free: its readers passed this barrier one head ago)
        uint8_t* dst = p.g.vcodes + ph * D * P + off;
        // thread: dim tid / 2, eight of the run's tokens (D * 2 threads)
        static_assert(kThreads == 2 * D, "two threads a dim");
        const int d = threadIdx.x >> 1, t0 = 8 * (threadIdx.x & 1);
        if (whole) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = st[(t0 + 4 * i) * kRow + d] | (st[(t0 + 4 * i + 1) * kRow + d] << 8) |
                       (st[(t0 + 4 * i + 2) * kRow + d] << 16) | (static_cast<uint32_t>(st[(t0 + 4 * i + 3) * kRow + d]) << 24);
            *reinterpret_cast<uint2*>(dst + static_cast<size_t>(d) * P + t0) = make_uint2(w[0], w[1]);
        } else {
            const int a = max(t0, first - base), b = min(t0 + 8, q.kv - base);
            for (int t = a; t < b; ++t) dst[static_cast<size_t>(d) * P + t] = st[t * kRow + d];
        }
    }
    if (__any_sync(0xffffffffu, open)) write_exact_rows<D>(p, live, h0, h1, c, row, page, off + tok);
}

template <int D>
cudaError_t launch_d(const PagedWriteParams& p, cudaStream_t s) {
    const int runs = static_cast<int>(paged_write_runs(p.g));
    const int64_t blocks = paged_write_blocks(p.g);
    // Heads of a block: two, which share the angles and overlap one's loads with
    // the other's work, four when those still fill the card three times (757
    // tokens x 48 heads x 128: one head 19.3 us, two 16.6, four 15.9, eight 19.7;
    // 64 single tokens x 8 heads: 5.8, 5.2, 5.4, 8.0).
    const int hpb = blocks * ((p.g.kv_heads + 3) / 4) >= 152 * 3 ? 4 : 2;
    dim3 grid(static_cast<unsigned>(blocks), (p.g.kv_heads + hpb - 1) / hpb);
    paged_write_kernel<D><<<grid, kRun * D / 8, 0, s>>>(p, runs, hpb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteParams& p, int D, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
