// rc_paged4_write.cu -- new tokens into the pages of the 4-bit cache: K turned at
// its positions, then K and V each quantised to E2M1 with one scale per 16 dims.
//   s = the least scale with max |x| <= 6 s,  code = E2M1 number nearest to x / s
// Bound by memory: bf16 K and V are read once, codes and scales written once.
// A block takes 16 cached tokens that lie side by side in a page (an aligned run,
// so that V's and the scales' pieces of 16 tokens are whole) and walks over some
// heads.  A token's row is held by D / 8 lanes with 8 dims each; two lanes have a
// scale's block.  The (cos, sin) of a token do not depend on the head: the block
// makes them once, in shared memory, from where each lane takes those of its dims.
// V's codes and all scales go through shared memory to be transposed (8 tokens x 8
// dims of codes are eight words whose nibbles change places).  Tokens of the run
// that are older than the call, or behind the sequence, keep their bits: the words
// that they share with new ones are read first.
// Everything is computed at 2^-8 of its value (folded into the turn's gain), so that
// no product of the largest bf16 numbers with the gain overflows.
// The codes and scales of K are those of the exact turn (to 2^-25 (|a| + |b|), what
// cos and sin leave): where an fp32 sum is too close to the middle between two codes,
// or a block's largest to the border between two scales, the warp's rows are summed
// again with twice the bits.
#include "rc_paged4.cuh"
#include "rc_turn_pair.cuh"

namespace rc {

namespace {

constexpr int kRun = kWriteRun;
constexpr int kMaxHeads = 4;        // of a block
constexpr float kDown = 0x1p-8f;

// How a lane comes by what its dims are paired with.
enum Partner : int {
    kInLane,  // neighbouring pairs, or nothing turns
    kVector,  // halves, the part and its half on a boundary of 8 dims: another lane's 8 dims
    kAnywhere // halves
};

// Byte of the least scale s with 6 s >= amax, cut to the top one; amax is 2^-8 of its value.
__device__ __forceinline__ uint32_t scale4_byte(float amax) {
    // a little less than amax / 6, rounded up to 8 bits: the scale or the one before it
    const float f = fminf(amax * (256.f / 6.f * (1.f - 0x1p-20f)), 10240.f);
    const uint32_t b = (static_cast<uint32_t>(__half_as_ushort(__float2half_ru(f))) + 0x7fu) >> 7;
    return b + (b < kTopScale4 && amax > scale4_value(b) * (6.f * kDown) ? 1u : 0u);
}

// Whether some number within `err` of amax has another scale than byte b.
__device__ __forceinline__ bool scale4_open(float amax, float err, uint32_t b) {
    return (b < kTopScale4 && amax + err > scale4_value(b) * (6.f * kDown)) ||
           (b > 0 && amax - err <= scale4_value(b - 1) * (6.f * kDown));
}

__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A quotient of numbers of few bits (8 by 4) that is off by some 2^-22 of itself, cut
// to 16 bits: one that lies on the middle between two codes is put there again, and
// no other one can get there.
__device__ __forceinline__ float to16bits(float q) { return __uint_as_float((__float_as_uint(q) + 0x80u) & ~0xffu); }

// The code by comparisons with the middles between codes, which are exact (a middle
// has 3 bits, a scale 4); s is 2^-8 of the scale.
__device__ __forceinline__ uint32_t codes8_exactly(const float (&y)[8], float s) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(y[i]);
        uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) + (a >= 3.5f * s) + (a > 5.f * s);
        c = s == 0.f ? 0u : c;
        w |= (c | (__float_as_uint(y[i]) >> 31 << 3)) << (4 * i);
    }
    return w;
}

// Where dim d turns: its pair, what it is paired with, the sign of that in the sum.
struct Role {
    int pair, partner;
    bool turns, upper;
};
__device__ __forceinline__ Role role_of(const RopeFormDev& f, int d) {
    Role r;
    const int rel = d - f.first, half = f.dims >> 1;
    r.turns = rel >= 0 && rel < f.dims;
    if (f.layout == RC_ROPE_HALVES) {
        r.upper = rel >= half;
        r.pair = r.upper ? rel - half : rel;
        r.partner = r.upper ? d - half : d + half;
    } else {
        r.upper = d & 1;
        r.pair = rel >> 1;
        r.partner = d ^ 1;
    }
    if (!r.turns) {
        r.pair = 0;
        r.partner = d;
    }
    return r;
}

// The exact sums of the lane's dims 8 c .. (rounded to odd) at 2^-8, from the row's K and the token's positions.
// (Out of line: what one warp of thousands needs costs the others little.)
__device__ __noinline__ void exact_sums(const Paged4WriteParams& p, const __nv_bfloat16* k, int row, int c, float* y) {
    const float g = p.form.gain * kDown;
    for (int j = 0; j < 8; ++j) {
        const int d = 8 * c + j;
        const Role r = role_of(p.form, d);
        const float a = __bfloat162float(k[d]), b = __bfloat162float(k[r.partner]);
        if (!r.turns) {
            y[j] = a * kDown;
            continue;
        }
        TurnPair t = turn_cos_sin_pair(__ldg(p.pos + p.form.axis[r.pair] * p.pos_stride + row), p.form.turns[r.pair]);
        const float2 hi = make_float2(__fmul_rn(t.hi.x, g), __fmul_rn(t.hi.y, g));
        const float2 lo = make_float2(__fmaf_rn(t.hi.x, g, -hi.x) + t.lo.x * g, __fmaf_rn(t.hi.y, g, -hi.y) + t.lo.y * g);
        y[j] = a == 0.f && b == 0.f ? 0.f : sum_exactly(a, hi.x, lo.x, r.upper ? b : -b, hi.y, lo.y);
    }
}

// Eight words, the nibbles of each a token's codes of eight dims, become eight words, the nibbles of each a dim's codes of
// eight tokens.
__device__ __forceinline__ void transpose_codes(uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i], b = w[i + 4];
        w[i] = __byte_perm(a, b, 0x5410);
        w[i + 4] = __byte_perm(a, b, 0x7632);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = (k & 1) | ((k & 2) << 1);
        const uint32_t a = w[i], b = w[i + 2];
        w[i] = __byte_perm(a, b, 0x6240);
        w[i + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t a = w[i], b = w[i + 1];
        w[i] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
        w[i + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
    }
}

__device__ __forceinline__ void open_bf16(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
// Whether a word holds a bf16 infinity or NaN.
__device__ __forceinline__ bool not_finite(const uint4& w) {
    auto half = [](uint32_t u) { return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u; };
    return half(w.x) || half(w.y) || half(w.z) || half(w.w);
}

template <int D, Partner PART>
__global__ void __launch_bounds__(kRun * D / 8, 512 / D) paged4_write_kernel(const __grid_constant__ Paged4WriteParams p, int runs, int heads_per_block) {
    constexpr int LANES = D / 8;  // of one token
    constexpr int kThreads = kRun * LANES;
    constexpr int NB = D / kBlock4;
    __shared__ float2 table[kRun * D / 2];
    __shared__ uint32_t scode[kMaxHeads][kRun][LANES + 1];             // V's codes
    __shared__ __align__(16) uint8_t sscale[kMaxHeads][2][NB][kRun];   // K's and V's scale bytes
    const int s = blockIdx.x / runs, run = blockIdx.x % runs;
    const Seq q = load_seq(p.g, s);
    if (q.n == 0) return;
    if (q.n > q.kv) {  // new tokens that the length does not count
        if (threadIdx.x == 0) flag_meta(p.g.status);
        return;
    }
    const int first = q.kv - q.n;                         // index of the first new token
    const int base = (first & ~(kRun - 1)) + run * kRun;  // index of the run's first token
    if (base >= q.kv) return;
    const int page = load_page(p.g, s, base >> p.g.page_shift);
    if (page < 0) return;
    const int P = 1 << p.g.page_shift, off = base & (P - 1);
    const int tok = threadIdx.x / LANES, c = threadIdx.x % LANES;
    const int index = base + tok;
    const bool live = index >= first && index < q.kv;
    const int row = q.q0 + (live ? index - first : 0);
    const int h0 = blockIdx.y * heads_per_block, h1 = min(p.g.kv_heads, h0 + heads_per_block);

    const Role mine = role_of(p.form, 8 * c);
    // (kVector: the lane's eight dims have one role)
    const int partner_at = PART == kVector ? mine.partner : 8 * c;
    const __nv_bfloat16* kr = p.K + row * p.k_stride;
    const __nv_bfloat16* vr = p.V + row * p.v_stride + c * 8;
    uint4 kw = make_uint4(0, 0, 0, 0), vw = kw, pw = kw;
    auto fetch = [&](int h) {
        kw = ldg_nc_na_v4(kr + static_cast<size_t>(h) * D + c * 8);
        if (PART == kVector) pw = __ldg(reinterpret_cast<const uint4*>(kr + static_cast<size_t>(h) * D + partner_at));
        vw = ldg_nc_na_v4(vr + static_cast<size_t>(h) * D);
    };
    if (live) fetch(h0);

    // the tokens' g (cos, sin) at 2^-8.  A sine of 0 says that nothing is rounded: where it is 0 only in fp32, it gets
    // its value, the angle itself
    const float g = p.form.gain * kDown;
    {
        const uint64_t* turns = param_address(p.form.turns);
        const uint8_t* axis = param_address(p.form.axis);
        const int pairs = p.form.dims >> 1;
        for (int i = threadIdx.x; i < kRun * pairs; i += kThreads) {
            const int t = i / pairs, k = i - t * pairs;
            if (base + t < first || base + t >= q.kv) continue;
            const int pos = __ldg(p.pos + axis[k] * p.pos_stride + q.q0 + base + t - first);
            float2 cs = turn_cos_sin(pos, turns[k]);
            if (cs.y == 0.f) {
                const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns[k];
                cs.y = cs.x * static_cast<float>(static_cast<int64_t>(frac << 1) >> 1) * 3.4061215e-19f;  // 2 pi / 2^64
            }
            table[t * (D / 2) + k] = make_float2(g * cs.x, g * cs.y);
        }
    }
    __syncthreads();
    float cs[8], sn[8];
    uint32_t exact = 0;  // dims whose sum is exact in fp32 (with a gain that is a power of two)
    {
        const bool plain = (__float_as_uint(p.form.gain) & 0x7fffffu) == 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const Role r = PART == kVector ? Role{mine.pair + j, 0, mine.turns, mine.upper} : role_of(p.form, 8 * c + j);
            cs[j] = kDown;
            sn[j] = 0.f;
            if (r.turns && live) {
                const float2 t = table[tok * (D / 2) + r.pair];
                cs[j] = t.x;
                sn[j] = r.upper ? t.y : -t.y;
            }
            exact |= (!r.turns || (sn[j] == 0.f && plain) ? 1u : 0u) << j;
        }
    }
    // lanes of the warp that have the token's row
    const uint32_t row_lanes = (LANES == 16 ? 0xffffu : 0xffu) << ((threadIdx.x & 31) & ~(LANES - 1));

    for (int h = h0; h < h1; ++h) {
        const int hl = h - h0;
        float x[8], xp[8], v[8];
        open_bf16(kw, x);
        open_bf16(vw, v);
        if (PART == kInLane) {
#pragma unroll
            for (int j = 0; j < 8; ++j) xp[j] = x[j ^ 1];
        } else if (PART == kVector) {
            open_bf16(pw, xp);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                xp[j] = live ? __bfloat162float(kr[static_cast<size_t>(h) * D + role_of(p.form, 8 * c + j).partner]) : 0.f;
        }
        const bool kbad = (__ballot_sync(0xffffffffu, not_finite(kw)) & row_lanes) != 0u;
        const bool vbad = (__ballot_sync(0xffffffffu, not_finite(vw)) & row_lanes) != 0u;
        if (live && h + 1 < h1) fetch(h + 1);  // the next head is on its way

        // K
        float y[8], reach = 0.f, amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = fmaf(x[j], cs[j], xp[j] * sn[j]);
            amax = fmaxf(amax, fabsf(y[j]));
            xp[j] = (exact >> j) & 1u ? 0.f : fabsf(x[j]) + fabsf(xp[j]);  // what its error is relative to
            reach = fmaxf(reach, xp[j]);
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        reach = fmaxf(reach, __shfl_xor_sync(0xffffffffu, reach, 1));
        uint32_t kb = scale4_byte(amax);
        // A sum is within 2^-21 g (|a| + |b|) of the exact one: cos and sin half an ulp of 1 each (2^-25), the gain and
        // three roundings 2^-24 each; the quotient by the scale adds 2^-22 of itself.
        const float slack = g * 0x1p-20f;
        bool again = reach > 0.f && scale4_open(amax, reach * slack, kb);
        const float inv = kb == 0u ? 0.f : reciprocal(scale4_value(kb) * kDown);
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float w = y[j] * inv, tol = xp[j] * (slack * inv);
            const float r = (exact >> j) & 1u ? to16bits(w) : w;
            lo[j] = r - tol;
            hi[j] = r + tol;
        }
        uint32_t kc = codes8(lo);
        again = (again || kc != codes8(hi)) && live && !kbad;
        if (__any_sync(0xffffffffu, again)) {
            float z[8];
            if (live && !kbad) exact_sums(p, kr + static_cast<size_t>(h) * D, row, c, z);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = 0.f;
            amax = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(z[j]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            kb = scale4_byte(amax);
            kc = codes8_exactly(z, scale4_value(kb) * kDown);
        }
        if (kbad) {
            kc = 0u;
            kb = 255u;
        }
        // V
        amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] *= kDown;
            amax = fmaxf(amax, fabsf(v[j]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        uint32_t vb = scale4_byte(amax);
        const float vinv = vb == 0u ? 0.f : reciprocal(scale4_value(vb) * kDown);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to16bits(v[j] * vinv);
        uint32_t vc = codes8(v);
        if (vbad) {
            vc = 0u;
            vb = 255u;
        }
        if (live) {
            const size_t at = ((static_cast<size_t>(page) * p.g.kv_heads + h) << p.g.page_shift) + off + tok;
            *reinterpret_cast<uint32_t*>(p.g.kcodes + at * (D / 2) + 4 * c) = kc;
        }
        scode[hl][tok][c] = vc;
        if ((c & 1) == 0) {
            sscale[hl][0][c >> 1][tok] = static_cast<uint8_t>(kb);
            sscale[hl][1][c >> 1][tok] = static_cast<uint8_t>(vb);
        }
    }
    __syncthreads();
    // tokens a .. b - 1 of the run are new
    const int a = max(0, first - base), b = min(kRun, q.kv - base);
    const int heads = h1 - h0;
    constexpr int kCodeJobs = 2 * LANES;  // of a head: 8 dims of 8 tokens each
    for (int i = threadIdx.x; i < heads * kCodeJobs; i += kThreads) {
        const int hl = i / kCodeJobs, c8 = i % LANES, t0 = 8 * ((i / LANES) & 1);
        const int m0 = max(a, t0) - t0, m1 = min(b, t0 + 8) - t0;  // new ones among the eight
        if (m1 <= m0) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            p.g.vcodes + ((static_cast<size_t>(page) * p.g.kv_heads + h0 + hl) * D + 8 * c8) * (P / 2) + (off + t0) / 2);
        const int step = P / 8;  // words between dims
        uint32_t w[8], old[8];
        const uint32_t mask = (m1 == 8 ? 0xffffffffu : (1u << (4 * m1)) - 1u) & ~((1u << (4 * m0)) - 1u);
#pragma unroll
        for (int j = 0; j < 8; ++j) old[j] = mask == 0xffffffffu ? 0u : dst[j * step];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = scode[hl][t0 + j][c8];
        transpose_codes(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j * step] = (w[j] & mask) | (old[j] & ~mask);
    }
    for (int i = threadIdx.x; i < heads * 2 * NB; i += kThreads) {
        const int hl = i / (2 * NB), which = (i / NB) & 1, nb = i % NB;
        uint8_t* dst = (which ? p.g.vscale : p.g.kscale) + ((static_cast<size_t>(page) * p.g.kv_heads + h0 + hl) * NB + nb) * P + off;
        const uint8_t* src = sscale[hl][which][nb];
        if (a == 0 && b == kRun)
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else
            for (int t = a; t < b; ++t) dst[t] = src[t];
    }
}

template <int D, Partner PART>
cudaError_t launch_part(const Paged4WriteParams& p, cudaStream_t s) {
    const int runs = static_cast<int>(paged_write_runs(p.g));
    const int64_t blocks = paged_write_blocks(p.g);
    const int hpb = blocks * ((p.g.kv_heads + 3) / 4) >= 152 * 3 ? 4 : 2;
    dim3 grid(static_cast<unsigned>(blocks), (p.g.kv_heads + hpb - 1) / hpb);
    paged4_write_kernel<D, PART><<<grid, kRun * D / 8, 0, s>>>(p, runs, hpb);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Paged4WriteParams& p, cudaStream_t s) {
    if (p.form.layout != RC_ROPE_HALVES || p.form.dims == 0) return launch_part<D, kInLane>(p, s);
    if (((p.form.first | (p.form.dims / 2)) & 7) == 0) return launch_part<D, kVector>(p, s);
    return launch_part<D, kAnywhere>(p, s);
}

}  // namespace

cudaError_t launch_paged4_write(const Paged4WriteParams& p, int D, cudaStream_t s) {
    return D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace rc
