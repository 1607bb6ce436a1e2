// rc_paged.cuh -- what the kernels over the paged cache share: parameter
// blocks, the sequence and page lookups (every index read from device memory
// is checked here before it is used), and the decode of E4M3 codes with E8M0
// scales to bf16.
#pragma once
#include "rc.h"
#include "rc_device.cuh"
#include "rc_internal.h"
#include "rc_paged_bounds.h"

namespace rc {

// Frequencies of the dimension pairs in turns, 64-bit fixed point.
struct RopePlanDev {
    uint64_t turns[kMaxHalfDim];
    uint8_t axis[kMaxHalfDim];
};

// What turns, in which layout, by which axes and frequencies (rc_rope_form).
struct RopeFormDev {
    uint64_t turns[RC_ROPE_MAX_HEAD_DIM / 2];
    uint8_t axis[RC_ROPE_MAX_HEAD_DIM / 2];
    int head_dim, first, dims, layout;
    float gain;
};

// A generic address of a kernel's (__grid_constant__) parameter bytes, whose
// origin the compiler does not see: lanes that read different entries of an
// array there go through the data cache together, where the constant bank
// would serve one address at a time (a chunk's write then took 22 us, not 15.6).
template <typename T>
__device__ __forceinline__ const T* param_address(const T* p) {
    asm volatile("mov.b64 %0, %0;" : "+l"(p));
    return p;
}

struct PagedParams {
    uint8_t* kcodes;
    uint8_t* vcodes;
    uint8_t* kscale;
    uint8_t* vscale;
    const int32_t* page_table;
    const int32_t* kv_len;
    const int32_t* q_start;
    int* status;
    int pages, kv_heads, page_shift;  // tokens of a page = 1 << page_shift (4 .. 7)
    int seqs, table_pages, tokens, max_new, max_kv;
};

// Device status word of the paged calls.
constexpr int kDevBadMeta = 301;

__device__ __forceinline__ void flag_meta(int* status) { atomicCAS(status, 0, kDevBadMeta); }

struct Seq {
    int q0, n, kv;  // first row, new tokens, cached tokens (new ones included)
};

// Sequence s as the metadata gives it; empty (and flagged) if it is out of the
// bounds that the host was told.
__device__ __forceinline__ Seq load_seq(const PagedParams& p, int s) {
    Seq q;
    q.kv = __ldg(p.kv_len + s);
    q.q0 = __ldg(p.q_start + s);
    const int end = __ldg(p.q_start + s + 1);
    if (paged_seq_ok(q.kv, q.q0, end, p.tokens, p.max_new, p.max_kv)) {
        q.n = end - q.q0;
    } else {
        flag_meta(p.status);
        q.q0 = q.n = q.kv = 0;
    }
    return q;
}

// Read-only loads that stay where they are written: the compiler would move a
// plain load made for the next step of a loop down to its use there.
__device__ __forceinline__ uint32_t ldg_early(const uint32_t* p) {
    uint32_t r;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}
__device__ __forceinline__ uint32_t ldg_early(const uint8_t* p) {
    uint32_t r;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(r) : "l"(p));
    return r;
}

// Whether a page table entry is a page of the pool; flagged if not.
__device__ __forceinline__ bool check_page(const PagedParams& p, int page) {
    if (paged_page_ok(page, p.pages)) return true;
    flag_meta(p.status);
    return false;
}

// Page of tokens [i P, i P + P) of sequence s, or -1 (flagged) if the table
// holds no page of the pool.  i P < kv_len <= table_pages P by load_seq.
__device__ __forceinline__ int load_page(const PagedParams& p, int s, int i) {
    const int page = __ldg(p.page_table + static_cast<size_t>(s) * p.table_pages + i);
    return check_page(p, page) ? page : -1;
}

// (cos, sin) of position * frequency: the product modulo one turn is exact in
// 64-bit integers; the nearest quarter turn is taken off as an integer, so
// what is left (at most an eighth) converts to fp32 with a relative error of
// 2^-24 before sincospi sees it.
__device__ __forceinline__ float2 turn_cos_sin(int pos, uint64_t turns) {
    const uint32_t frac = static_cast<uint32_t>((static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns) >> 32);
    const uint32_t quad = (frac + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(frac - (quad << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // half turns: rest / 2^31
    const bool odd = quad & 1u;
    const float cc = odd ? s : c, ss = odd ? c : s;
    return make_float2((quad == 1u || quad == 2u) ? -cc : cc, (quad & 2u) ? -ss : ss);
}

// ---------------------------------------------------------------- decode
// An E4M3 byte s eeee mmm put at s 0000 eeee mmm 0000 of a bf16 word is its
// value times 2^-120, subnormals included (both formats are then subnormal or
// normal together); one bf16 multiply by 2^120 times the scale, 2^(b - 7) for
// an E8M0 byte b, makes it exact.  A word of four codes c0..c3 (c0 in the low
// byte) gives the pairs (c0, c2) and (c1, c3): two shifts and masks each,
// where neighbouring codes would need a byte permute more.
__device__ __forceinline__ uint32_t codes02(uint32_t w) {
    return ((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t codes13(uint32_t w) {
    return (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
}
// The pairs (c0, c1) and (c2, c3): the bytes are first put at the tops of the halves.
__device__ __forceinline__ uint32_t codes_apart(uint32_t t) { return (t & 0x80008000u) | ((t >> 4) & 0x07f007f0u); }
__device__ __forceinline__ uint32_t codes01(uint32_t w) { return codes_apart(__byte_perm(w, 0u, 0x1404)); }
__device__ __forceinline__ uint32_t codes23(uint32_t w) { return codes_apart(__byte_perm(w, 0u, 0x3424)); }
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// bf16 factor 2^(b + 120 - 127) of scale byte b, in both halves; bytes over
// 134 (255: a row that is not finite) give infinity, which makes a zero code
// NaN and any other code infinite.
__device__ __forceinline__ uint32_t scale_factor(uint32_t b) {
    const uint32_t f = min(b + 120u, 255u) << 7;
    return f | (f << 16);
}
// The factors of scale bytes (0, 2) and (1, 3) of a word.
__device__ __forceinline__ uint32_t scale_factor2(uint32_t two) {  // bytes in bits 0..7 and 16..23
    return __vminu2(two + 0x00780078u, 0x00ff00ffu) << 7;
}
__device__ __forceinline__ uint32_t factors02(uint32_t w) { return scale_factor2(w & 0x00ff00ffu); }
__device__ __forceinline__ uint32_t factors13(uint32_t w) { return scale_factor2((w >> 8) & 0x00ff00ffu); }

// The fp32 value of E8M0 byte `byte` of a word: 2^(b - 127), and NaN (or, for
// bytes that no row here has, 2^127 and up) for 255.
__device__ __forceinline__ float e8m0_float(uint32_t w, int byte) {
    const uint32_t b = (w >> (8 * byte)) & 0xffu;
    return __uint_as_float(b == 255u ? 0x7fc00000u : b << 23);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 codes as bf16, in the order (0, 2), (1, 3) of each four, with the factors
// of the pairs.
__device__ __forceinline__ void put16(uint8_t* lo, uint8_t* hi, const uint4& w, const uint32_t (&f)[8]) {
    *reinterpret_cast<uint4*>(lo) = make_uint4(bf2_mul(codes02(w.x), f[0]), bf2_mul(codes13(w.x), f[1]),
                                               bf2_mul(codes02(w.y), f[2]), bf2_mul(codes13(w.y), f[3]));
    *reinterpret_cast<uint4*>(hi) = make_uint4(bf2_mul(codes02(w.z), f[4]), bf2_mul(codes13(w.z), f[5]),
                                               bf2_mul(codes02(w.w), f[6]), bf2_mul(codes13(w.w), f[7]));
}

// E8M0 byte of a row's scale from its largest magnitude: the smallest e with
// amax <= 448 * 2^e = 1.75 * 2^(e + 8), cut to -124 .. 7; 0 for a row of zeros.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int k = static_cast<int>(u >> 23) - 127;
    const int e = k - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax == 0.f ? 0 : max(-124, min(7, e));
}

// D += A B, A a 16 x 16 row-major fragment, B 16 x 8, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit numbers transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Four E4M3 codes (code 0 in the low byte) as fp16, exactly: pairs (0, 1), (2, 3).
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// The e of the 2^e that a query row is divided by for fp16: 14 <= log2(amax) - e < 15,
// e kept where 2^e and 2^-e are normal numbers; rows of zeros, and rows that are not
// finite, are taken as they are.
__device__ __forceinline__ int row_exponent(float amax) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14;
    return amax > 0.f && amax <= 3.4028235e38f ? max(-126, min(126, e)) : 0;
}

// Query rows as the B operand of S^T = K Q^T with K's codes as fp16: 8 rows a
// tile, row lane / 4 of tile r at row[r].  Each row is divided by a power of two
// that puts its largest magnitude in [2^14, 2^15), so that bf16's 8 bits are
// exact in fp16 down to 2^-32 of it (what is smaller loses bits that are nothing
// beside the row's largest).  The lane (t = lane % 4) has RUN neighbouring dims at a
// time: product c * RUN / 4 + i holds dims RUN (t + 4 c) + 4 i + {0, 1} and + {2, 3},
// as codes_f16 gives them.
// scale[r][x]: that power times `factor` for row 2 t + x of tile r, the rows
// whose scores the lane gets.
template <int D, int NR, int RUN = 16>
__device__ __forceinline__ void query_tile_f16(const __nv_bfloat16* const (&row)[NR], const bool (&live)[NR], float factor,
                                               uint32_t (&qb)[NR][D / 16][2], float (&scale)[NR][2]) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        uint32_t w[D / 8];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 8; c += 4) {  // eight dims
            uint4 a = make_uint4(0, 0, 0, 0);
            if (live[r]) a = __ldg(reinterpret_cast<const uint4*>(row[r] + RUN * (t + 4 * (2 * c / RUN)) + 2 * c % RUN));
            const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[c + i] = x[i];
                amax = max3(amax, fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u)));
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = row_exponent(amax);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float mine = factor * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
        for (int x = 0; x < 2; ++x) scale[r][x] = __shfl_sync(0xffffffffu, mine, 4 * (2 * t + x));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t v = w[2 * k + x];
                __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
                qb[r][k][x] = *reinterpret_cast<uint32_t*>(&h);
            }
    }
}

struct PagedWriteParams {
    PagedParams g;
    RopePlanDev rope;
    const __nv_bfloat16* K;
    const __nv_bfloat16* V;
    const int32_t* pos;
    int64_t k_stride, v_stride, pos_stride;
};

struct Paged4WriteParams {
    PagedParams g;
    RopeFormDev form;  // dims 0: K is stored as it comes
    const __nv_bfloat16* K;
    const __nv_bfloat16* V;
    const int32_t* pos;
    int64_t k_stride, v_stride, pos_stride;
};

struct PagedAttnParams {
    PagedParams g;
    const __nv_bfloat16* q;
    int64_t q_stride;
    __nv_bfloat16* out;
    int64_t out_stride;
    float* lse;        // may be nullptr
    int heads, group;  // query heads, query heads of one KV head
    int causal;
    float sm_log2;     // log2(e) / sqrt(head_dim)
    int split_tokens;  // cached tokens of one split (a multiple of 256)
    int splits;        // splits of a sequence of max_kv tokens
    int row_tiles;     // kernels with row tiles: those of the longest sequence that they take
    int few;           // tcgen05 kernels: sequences with up to so many rows a KV head are another kernel's (0: none is)
    int most;          // 4-bit kernels of few rows: so are those with more than so many
    float* part;       // workspace: partial results
    int* counters;     // workspace: arrivals of the splits, all zero between calls
    uint64_t wait_ns;
};

struct PagedScoreParams {
    PagedParams g;
    const __nv_bfloat16* q;
    int64_t q_stride;
    const float* lse;
    const float* scores;
    float* out;
    int64_t score_stride;
    int heads, group, causal;
    float sm_log2;
    uint64_t wait_ns;
};

struct PagedEvictParams {
    PagedParams g;
    const float* scores;
    int64_t score_stride;
    int keep, recent, dst_pages;
    const int32_t* dst_table;
    int32_t* kept;
    int32_t* kv_len_out;
    float* scores_out;  // may be nullptr
};

struct RopeAxesParams {
    RopePlanDev rope;
    const void* x;
    void* out;
    int64_t x_stride, out_stride, pos_stride, n;
    const int32_t* pos;
    int heads, inverse;
};

struct RopeFormParams {
    RopeFormDev form;
    const void* x;
    void* out;
    int64_t x_stride, out_stride, pos_stride, n;
    const int32_t* pos;
    int heads, back;
};

// Blocks in the x of a grid, from what the host was told.
constexpr int kWriteRun = 16;    // cached tokens of a block of the write: the alignment of a V row's piece
constexpr int kAttendRows = 256; // query rows of a block of the tcgen05 attention
inline int64_t paged_write_runs(const PagedParams& g) {  // that max_new tokens can touch, wherever the first one lies
    return (static_cast<int64_t>(g.max_new) + kWriteRun - 2) / kWriteRun + 1;
}
inline int64_t paged_write_blocks(const PagedParams& g) { return g.seqs * paged_write_runs(g); }
inline int64_t paged_attend_blocks(const PagedParams& g, int64_t rows) {
    return (rows + kAttendRows - 1) / kAttendRows * g.seqs * g.kv_heads;
}

cudaError_t launch_rope_axes(const RopeAxesParams& p, int D, int dtype, cudaStream_t s);
cudaError_t launch_rope_form(const RopeFormParams& p, int dtype, cudaStream_t s);
cudaError_t launch_paged_write(const PagedWriteParams& p, int D, cudaStream_t s);
cudaError_t launch_paged_attention(PagedAttnParams& p, int D, size_t part_floats, int max_counters, cudaStream_t s);
cudaError_t launch_paged_tc(PagedAttnParams& p, int D, size_t part_floats, cudaStream_t s);
cudaError_t launch_paged_scores(const PagedScoreParams& p, int D, cudaStream_t s);
cudaError_t launch_paged_scores_tc(const PagedScoreParams& p, int D, cudaStream_t s);
cudaError_t launch_paged_evict(const PagedEvictParams& p, int D, cudaStream_t s);
cudaError_t launch_paged4_write(const Paged4WriteParams& p, int D, cudaStream_t s);
cudaError_t launch_paged4_attention(PagedAttnParams& p, int D, size_t part_floats, cudaStream_t s);
cudaError_t launch_paged4_tc(PagedAttnParams& p, int D, size_t part_floats, cudaStream_t s);

}  // namespace rc
