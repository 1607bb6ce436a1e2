// rc_paged4_write.cu -- new tokens into the pages of the 4-bit cache: K turned at
// its positions, then K and V each quantised to E2M1 with one scale per 16 dims.
//   s = the least scale with max |x| <= 6 s,  code = E2M1 number nearest to x / s
// Bf16 K and V are read once, codes and scales written once: 757 tokens x 48 heads x 128
// are 24 MB, 3.6 us at the copy rate, and take 13.0 us as pairs on three axes, 13.5 as
// halves, 15.0 as halves of 36 dims, 11.6 without a turn.  Memory does not bound it (DRAM
// at 15 % of its peak) and issue alone does not either (54 % of the cycles, 408
// instructions a warp and head, all counted): the 392 blocks are less than one wave with
// 4.6 warps a scheduler, and the fullest scheduler has 1.24 times the mean's work.
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
// or a block's largest to the border between two scales, it is (or they are) summed
// again with twice the bits.
#include "rc_paged4.cuh"
#include "rc_turn_pair.cuh"

namespace rc {

namespace {

constexpr int kRun = kWriteRun;
constexpr int kMaxHeads = 6;        // of a block
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

// The codes of quotients by s, r its reciprocal: the remainder of the first product is added in, so that a quotient that
// is a number of fp32 is that number.  (What lies on the middle between two codes stays there; other quotients of numbers
// of 8 bits by one of 4 are 2^-9 of themselves away from it.)  Taken with the other sign, a zero keeps its own.
__device__ __forceinline__ uint32_t codes8_of_quotients(const float2 (&x)[4], float s, float r) {
    const float2 s2 = make_float2(s, s), r2 = make_float2(-r, -r);
    float w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 q = mul2(x[j], r2), u = fma2(fma2(q, s2, x[j]), r2, q);
        w[2 * j] = u.x;
        w[2 * j + 1] = u.y;
    }
    return codes8(w) ^ 0x88888888u;
}

// The code by comparisons with the middles between codes, which are exact (a middle
// has 3 bits, a scale 4); s is 2^-8 of the scale.
__device__ __forceinline__ uint32_t code_exactly(float y, float s) {
    const float a = fabsf(y);
    const uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) + (a >= 3.5f * s) + (a > 5.f * s);
    return (s == 0.f ? 0u : c) | (__float_as_uint(y) >> 31 << 3);
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

// The exact sum of dim d (rounded to odd) at 2^-8, from the row's K and the token's positions.  (Out of line: what some
// values of a hundred thousand need costs the others little.)
__device__ __noinline__ float exact_sum(const Paged4WriteParams& p, const __nv_bfloat16* k, int row, int d) {
    const float g = p.form.gain * kDown;
    const Role r = role_of(p.form, d);
    const float a = __bfloat162float(k[d]), b = __bfloat162float(k[r.partner]);
    if (!r.turns) return a * kDown;
    const TurnPair t = turn_cos_sin_pair(__ldg(p.pos + p.form.axis[r.pair] * p.pos_stride + row), p.form.turns[r.pair]);
    const float2 hi = make_float2(__fmul_rn(t.hi.x, g), __fmul_rn(t.hi.y, g));
    const float2 lo = make_float2(__fmaf_rn(t.hi.x, g, -hi.x) + t.lo.x * g, __fmaf_rn(t.hi.y, g, -hi.y) + t.lo.y * g);
    return a == 0.f && b == 0.f ? 0.f : sum_exactly(a, hi.x, lo.x, r.upper ? b : -b, hi.y, lo.y);
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

__device__ __forceinline__ void open_bf16(const uint4& w, float2 (&x)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
// The larger of two pairs of numbers of 16 bits, each.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The largest magnitude of eight bf16 numbers, as the bits of one: infinities and NaNs are above every number.
__device__ __forceinline__ uint32_t largest_bits(const uint4& w) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = max_u16x2(max_u16x2(w.x & kAbs, w.y & kAbs), max_u16x2(w.z & kAbs, w.w & kAbs));
    return max(m & 0xffffu, m >> 16);
}
constexpr uint32_t kInfBits = 0x7f80u;

template <int D, Partner PART>
__global__ void __launch_bounds__(kRun * D / 8, 384 / D) paged4_write_kernel(const __grid_constant__ Paged4WriteParams p, int runs, int heads_per_block) {
    constexpr int LANES = D / 8;  // of one token
    constexpr int kThreads = kRun * LANES;
    constexpr int NB = D / kBlock4;
    constexpr int kCodeJobs = LANES;  // of a head: V's codes of 8 dims of the run each
    __shared__ float2 table[kRun * D / 2];
    __shared__ uint32_t scode[kMaxHeads][kRun][LANES + 1];             // V's codes
    __shared__ uint2 sold[8][kMaxHeads * kCodeJobs];                   // the words that they go into, of a run that is not all new
    __shared__ __align__(16) uint8_t sscale[kMaxHeads][2][NB][kRun];   // K's and V's scale bytes
    __shared__ __align__(16) uint16_t skey[PART == kAnywhere ? kThreads * 8 : 1];  // K's rows
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
    const int entry = __ldg(p.g.page_table + static_cast<size_t>(s) * p.g.table_pages + (base >> p.g.page_shift));
    const int P = 1 << p.g.page_shift, off = base & (P - 1);
    const int tok = threadIdx.x / LANES, c = threadIdx.x % LANES, lane = threadIdx.x & 31;
    const int index = base + tok;
    const bool live = index >= first && index < q.kv;
    const int row = q.q0 + (live ? index - first : 0);
    const int h0 = blockIdx.y * heads_per_block, h1 = min(p.g.kv_heads, h0 + heads_per_block), heads = h1 - h0;
    // tokens a .. b - 1 of the run are new
    const int a = max(0, first - base), b = min(kRun, q.kv - base);

    const __nv_bfloat16* kr = p.K + row * p.k_stride;
    const __nv_bfloat16* vr = p.V + row * p.v_stride;
    struct Words {
        uint4 k, v;
    };
    auto fetch = [&](Words& w, int h) {
        w.k = ldg_nc_na_v4(kr + static_cast<size_t>(h) * D + c * 8);
        w.v = ldg_nc_na_v4(vr + static_cast<size_t>(h) * D + c * 8);
    };
    Words even{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, odd = even;
    if (live) {
        fetch(even, h0);
        if (heads > 1) fetch(odd, h0 + 1);
    }

    // the tokens' g (cos, sin) at 2^-8, by the lanes that have the token's row.  A sine of 0 says that nothing is rounded:
    // where it is 0 only in fp32, it gets its value, the angle itself
    const float g = p.form.gain * kDown;
    const int pairs = p.form.dims >> 1;
    {
        constexpr int kEach = D / 2 / LANES;
        const uint64_t* turns = param_address(p.form.turns);
        const uint8_t* axis = param_address(p.form.axis);
        int pos[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            pos[i] = live && c + LANES * i < pairs ? __ldg(p.pos + axis[c + LANES * i] * p.pos_stride + row) : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = c + LANES * i;
            if (!live || k >= pairs) continue;
            float2 cs = turn_cos_sin(pos[i], turns[k]);
            if (cs.y == 0.f) {
                const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos[i])) * turns[k];
                cs.y = cs.x * static_cast<float>(static_cast<int64_t>(frac << 1) >> 1) * 3.4061215e-19f;  // 2 pi / 2^64
            }
            table[tok * (D / 2) + k] = make_float2(g * cs.x, g * cs.y);
        }
    }
    const int page = check_page(p.g, entry) ? entry : -1;
    if (page < 0) return;
    const size_t at0 = static_cast<size_t>(page) * p.g.kv_heads + h0;  // of the first head
    auto codes_of = [&](int job) {  // the first of its eight pairs of words, P / 16 pairs apart
        return reinterpret_cast<uint2*>(p.g.vcodes + ((at0 + job / kCodeJobs) * D + 8 * (job % kCodeJobs)) * (P / 2) + off / 2);
    };
    if (b - a < kRun)
        for (int i = threadIdx.x; i < heads * kCodeJobs; i += kThreads)
#pragma unroll
            for (int j = 0; j < 8; ++j) cp_async8(&sold[j][i], codes_of(i) + j * (P / 16));
    __syncwarp();
    float2 cs[4], sn[4];
    uint32_t partner[4] = {0, 0, 0, 0};  // kAnywhere: where in the row's 16-bit numbers, two a word
    const bool plain = (__float_as_uint(p.form.gain) & 0x7fffffu) == 0u;  // a power of two
    uint32_t exact = 0;  // the dims whose sums are exact in fp32, four bits each
    const Role mine = role_of(p.form, 8 * c);
    {
        float cc[8], ss[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // (kVector: the lane's eight dims have one role)
            const Role r = PART == kVector ? Role{mine.pair + j, 0, mine.turns, mine.upper} : role_of(p.form, 8 * c + j);
            cc[j] = kDown;
            ss[j] = 0.f;
            if (r.turns && live) {
                const float2 t = table[tok * (D / 2) + r.pair];
                cc[j] = t.x;
                ss[j] = r.upper ? t.y : -t.y;
            }
            if (!r.turns || (plain && ss[j] == 0.f)) exact |= 0xfu << (4 * j);
            if (PART == kAnywhere) partner[j / 2] |= static_cast<uint32_t>(r.partner) << (16 * (j & 1));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cs[j] = make_float2(cc[2 * j], cc[2 * j + 1]);
            sn[j] = make_float2(ss[2 * j], ss[2 * j + 1]);
        }
    }
    const bool some_exact = __any_sync(0xffffffffu, exact != 0u), all_exact = __all_sync(0xffffffffu, exact == 0xffffffffu);
    // lanes of the warp that have the token's row, and the one that has what this one's dims are paired with
    const uint32_t row_lanes = (LANES == 16 ? 0xffffu : 0xffu) << (lane & ~(LANES - 1));
    const int partner_lane = (lane & ~(LANES - 1)) + (PART == kVector ? mine.partner / 8 : c);

    auto head = [&](int h, Words& words) {
        const int hl = h - h0;
        const uint4 kw = words.k, vw = words.v;
        float2 x[4], xp[4];
        open_bf16(kw, x);
        const uint32_t kmost = largest_bits(kw), vmost = largest_bits(vw);
        uint32_t pmost = kmost;  // of what the dims are paired with
        if (PART == kInLane) {
#pragma unroll
            for (int j = 0; j < 4; ++j) xp[j] = make_float2(x[j].y, x[j].x);
        } else if (PART == kVector) {
            uint4 w;
            w.x = __shfl_sync(0xffffffffu, kw.x, partner_lane);
            w.y = __shfl_sync(0xffffffffu, kw.y, partner_lane);
            w.z = __shfl_sync(0xffffffffu, kw.z, partner_lane);
            w.w = __shfl_sync(0xffffffffu, kw.w, partner_lane);
            open_bf16(w, xp);
            pmost = __shfl_sync(0xffffffffu, kmost, partner_lane);
        } else {
            __syncwarp();
            *reinterpret_cast<uint4*>(skey + 8 * threadIdx.x) = kw;
            __syncwarp();
            const uint16_t* staged = skey + tok * D;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                xp[j] = make_float2(__uint_as_float(static_cast<uint32_t>(staged[partner[j] & 0xffffu]) << 16),
                                    __uint_as_float(static_cast<uint32_t>(staged[partner[j] >> 16]) << 16));
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) pmost = max(pmost, __shfl_xor_sync(0xffffffffu, pmost, o));
        }
        const bool kbad = (__ballot_sync(0xffffffffu, kmost >= kInfBits) & row_lanes) != 0u;
        const bool vbad = (__ballot_sync(0xffffffffu, vmost >= kInfBits) & row_lanes) != 0u;
        // K
        float2 y[4];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = fma2(x[j], cs[j], mul2(xp[j], sn[j]));
            amax = max3(amax, fabsf(y[j].x), fabsf(y[j].y));
        }
        // A sum is within 2^-22 g (|a| + |b|) of the exact one (cos and sin half an ulp of 1 each, 2^-25, and three
        // roundings of 2^-24), and 2^-23 more with a gain that is rounded; the quotient by the scale adds 2^-22 of itself:
        // 2^-21 of g (|a| + |b|), or 1.25 times that.
        const float slack = g * (plain ? 0x1p-21f : 0x1.4p-21f);
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const float err = exact == 0xffffffffu ? 0.f : __uint_as_float(max(kmost, pmost) << 16) * (2.f * slack);  // (at most, of all)
        float err2 = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, 1));
        if (some_exact) {  // a block whose largest is one of its exact sums is not open
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!((exact >> (4 * j)) & 1u)) most = fmaxf(most, fabsf(j & 1 ? y[j / 2].y : y[j / 2].x));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            if (most + err2 < amax) err2 = 0.f;
        }
        uint32_t kb = scale4_byte(amax);
        const __nv_bfloat16* keys = kr + static_cast<size_t>(h) * D;
        bool open = live && !kbad && err2 > 0.f && scale4_open(amax, err2, kb);
        if (__any_sync(0xffffffffu, open)) {  // the scale may be another: the sums that may be the block's largest, taken again
            const bool other = __shfl_xor_sync(0xffffffffu, open ? 1 : 0, 1) != 0;  // (all lanes, before anything is decided)
            open = open || other;
            uint32_t may = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) may |= (fabsf(j & 1 ? y[j / 2].y : y[j / 2].x) >= amax - 2.f * err2 ? 1u : 0u) << j;
            float most = 0.f;
            while (open && may != 0u) {
                most = fmaxf(most, fabsf(exact_sum(p, keys, row, 8 * c + __ffs(may) - 1)));
                may &= may - 1;
            }
            __syncwarp();
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            if (open) kb = scale4_byte(most);
        }
        const float scale = scale4_value(kb) * kDown, inv = kb == 0u ? 0.f : reciprocal(scale);
        uint32_t kc = 0u, unsure = 0u;
        if (!all_exact) {
            float lo[8], hi[8];
            const float reach = slack * inv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 w = mul2(y[j], make_float2(inv, inv));
                const float2 tol = mul2(make_float2(fabsf(x[j].x) + fabsf(xp[j].x), fabsf(x[j].y) + fabsf(xp[j].y)), make_float2(reach, reach));
                const float2 u = add2(w, tol);
                lo[2 * j] = w.x - tol.x;
                lo[2 * j + 1] = w.y - tol.y;
                hi[2 * j] = u.x;
                hi[2 * j + 1] = u.y;
            }
            kc = codes8(lo);
            unsure = (kc ^ codes8(hi)) & ~exact;
        }
        if (some_exact) kc = (kc & ~exact) | (codes8_of_quotients(y, scale, inv) & exact);
        if (!live || kbad) unsure = 0u;
        while (unsure != 0u) {
            const int j = (__ffs(unsure) - 1) >> 2;
            unsure &= ~(0xfu << (4 * j));
            kc = (kc & ~(0xfu << (4 * j))) | code_exactly(exact_sum(p, keys, row, 8 * c + j), scale) << (4 * j);
        }
        __syncwarp();
        if (kbad) {
            kc = 0u;
            kb = 255u;
        }
        // V
        const uint32_t vtop = max(vmost, __shfl_xor_sync(0xffffffffu, vmost, 1));
        uint32_t vb = scale4_byte(__uint_as_float(vtop << 16) * kDown);
        const float vscale = scale4_value(vb), vinv = vb == 0u ? 0.f : reciprocal(vscale);
        float2 v[4];
        open_bf16(vw, v);
        if (live && h + 2 < h1) fetch(words, h + 2);  // the head after the next
        uint32_t vc = codes8_of_quotients(v, vscale, vinv);
        if (vbad) {
            vc = 0u;
            vb = 255u;
        }
        if (live) *reinterpret_cast<uint32_t*>(p.g.kcodes + (((at0 + hl) << p.g.page_shift) + off + tok) * (D / 2) + 4 * c) = kc;
        scode[hl][tok][c] = vc;
        if ((c & 1) == 0) {
            sscale[hl][0][c >> 1][tok] = static_cast<uint8_t>(kb);
            sscale[hl][1][c >> 1][tok] = static_cast<uint8_t>(vb);
        }
    };
#pragma unroll 1
    for (int h = h0; h < h1; h += 2) {
        head(h, even);
        if (h + 1 < h1) head(h + 1, odd);
    }
    cp_async_wait_all();
    __syncthreads();
    for (int i = threadIdx.x; i < heads * kCodeJobs; i += kThreads) {
        const int hl = i / kCodeJobs, c8 = i % kCodeJobs;
        uint2* dst = codes_of(i);
        const int step = P / 16;  // pairs of words between dims
        uint32_t w[2][8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[half][j] = scode[hl][8 * half + j][c8];
            transpose_codes(w[half]);
        }
        if (b - a == kRun) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[j * step] = make_uint2(w[0][j], w[1][j]);
        } else {
            const uint64_t mask = (b == kRun ? ~0ull : (1ull << (4 * b)) - 1ull) & ~((1ull << (4 * a)) - 1ull);
            const uint32_t m0 = static_cast<uint32_t>(mask), m1 = static_cast<uint32_t>(mask >> 32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint2 old = sold[j][i];
                dst[j * step] = make_uint2((w[0][j] & m0) | (old.x & ~m0), (w[1][j] & m1) | (old.y & ~m1));
            }
        }
    }
    for (int i = threadIdx.x; i < heads * 2 * NB; i += kThreads) {
        const int hl = i / (2 * NB), which = (i / NB) & 1, nb = i % NB;
        uint8_t* dst = (which ? p.g.vscale : p.g.kscale) + ((at0 + hl) * NB + nb) * P + off;
        const uint8_t* src = sscale[hl][which][nb];
        if (a == 0 && b == kRun)
            *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        else
            for (int t = a; t < b; ++t) dst[t] = src[t];
    }
}

// Heads of a block: six, which share the angles, where those still give each SM two blocks: 4 x 2,000 tokens x 8 heads x
// 128 take 25.2 us with two, 21.8 with four, 20.0 with six, 23.0 with eight; 757 x 48 heads 15.8, 13.9, 13.1 and 12.9; 256
// single tokens x 8 heads 12.9, 12.3, 11.1 and 11.6.  Else two, for the call's latency: 64 single tokens x 8 heads 5.7 us
// with two, 7.7 with six; one token 4.6 and 7.4.
template <int D, Partner PART>
cudaError_t launch_part(const Paged4WriteParams& p, cudaStream_t s) {
    const int runs = static_cast<int>(paged_write_runs(p.g));
    const int64_t blocks = paged_write_blocks(p.g);
    const int hpb = blocks * ((p.g.kv_heads + kMaxHeads - 1) / kMaxHeads) >= 152 * 2 ? kMaxHeads : 2;
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
