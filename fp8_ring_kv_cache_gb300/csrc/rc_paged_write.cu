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
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kRun = 16;  // tokens of a block: the alignment of a V row's piece

// The lane's 8 values quantised with the row's scale; returns the scale byte.
template <int LANES>
__device__ __forceinline__ uint32_t quantise(const float (&x)[8], uint2& codes) {
    // the largest magnitude as bits: infinities and NaNs are above every number
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = top >= 0x7f800000u;
    const float amax = __uint_as_float(top);
    const int e = scale_exponent(amax);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e in -124 .. 7: exact
    codes = make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16),
                       e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16));
    if (bad) codes = make_uint2(0u, 0u);
    return bad ? 255u : static_cast<uint32_t>(e + 127);
}

template <int D>
__global__ void __launch_bounds__(kRun* D / 8) paged_write_kernel(const __grid_constant__ PagedWriteParams p, int runs, int heads_per_block) {
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

    float2 cs[4];
    const uint64_t* turns = param_address(p.rope.turns) + 4 * c;
    const uint32_t axes = *reinterpret_cast<const uint32_t*>(param_address(p.rope.axis) + 4 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        cs[i] = turn_cos_sin(__ldg(p.pos + ((axes >> (8 * i)) & 0xffu) * p.pos_stride + row), turns[i]);
    const __nv_bfloat16* kr = p.K + row * p.k_stride + c * 8;
    const __nv_bfloat16* vr = p.V + row * p.v_stride + c * 8;
    const int h0 = blockIdx.y * heads_per_block, h1 = min(p.g.kv_heads, h0 + heads_per_block);
    uint4 kw = make_uint4(0, 0, 0, 0), vw = kw;
    if (live) {
        kw = ldg_nc_na_v4(kr + static_cast<size_t>(h0) * D);
        vw = ldg_nc_na_v4(vr + static_cast<size_t>(h0) * D);
    }
    for (int h = h0; h < h1; ++h) {
        float k[8], v[8];
        const uint32_t ki[4] = {kw.x, kw.y, kw.z, kw.w}, vi[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rotate_pair(__uint_as_float(ki[i] << 16), __uint_as_float(ki[i] & 0xFFFF0000u), cs[i].x, cs[i].y, k[2 * i],
                        k[2 * i + 1]);
            v[2 * i] = __uint_as_float(vi[i] << 16);
            v[2 * i + 1] = __uint_as_float(vi[i] & 0xFFFF0000u);
        }
        if (live && h + 1 < h1) {  // the next head is on its way
            kw = ldg_nc_na_v4(kr + static_cast<size_t>(h + 1) * D);
            vw = ldg_nc_na_v4(vr + static_cast<size_t>(h + 1) * D);
        }
        uint2 kc, vc;
        const uint32_t kb = quantise<LANES>(k, kc), vb = quantise<LANES>(v, vc);
        const size_t ph = static_cast<size_t>(page) * p.g.kv_heads + h;
        uint8_t* st = stage[(h - h0) & 1];
        if (live) {
            *reinterpret_cast<uint2*>(p.g.kcodes + (ph * P + off + tok) * D + c * 8) = kc;
            *reinterpret_cast<uint2*>(st + tok * kRow + c * 8) = vc;
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
}

template <int D>
cudaError_t launch_d(const PagedWriteParams& p, cudaStream_t s) {
    // runs that max_new tokens can touch, wherever the first one lies
    const int runs = (p.g.max_new + kRun - 2) / kRun + 1;
    const int64_t blocks = static_cast<int64_t>(p.g.seqs) * runs;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    // Heads of a block: one while that does not fill the card three times, then
    // up to four, which share the angles and overlap a head's loads with the one
    // before (757 tokens x 48 heads x 128: one head 15.6 us, two 13.6, four 13.1,
    // eight 16.6; 64 single tokens x 8 heads: 4.9, 4.6, 4.8, 6.9).
    int hpb = 1;
    while (hpb < 4 && blocks * ((p.g.kv_heads + 2 * hpb - 1) / (2 * hpb)) >= 152 * 3) hpb *= 2;
    dim3 grid(static_cast<unsigned>(blocks), (p.g.kv_heads + hpb - 1) / hpb);
    paged_write_kernel<D><<<grid, kRun * D / 8, 0, s>>>(p, runs, hpb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteParams& p, int D, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
