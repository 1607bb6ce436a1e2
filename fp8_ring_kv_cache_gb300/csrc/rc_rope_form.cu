// rc_rope_form.cu -- rotary positions in other forms than rc_rope_axes'
// (rc_rope_turn): neighbouring pairs or halves, a part of the head, a gain;
// forward, or back (the gradient: the turn's transpose with the same gain).
//   (a, b) -> g (a cos - b sin, a sin + b cos) per pair, the other dims copied
// Bound by memory: every value is read and written once.  A block computes its
// tokens' g (cos, sin) once into shared memory, where all heads read them.  A
// thread turns a piece of V neighbouring dims and, for halves, the piece half a
// part further on that they are paired with: V is the most (16 bytes, 32 of
// neighbouring pairs) that divides the part's start and half, so that every
// piece lies on V's boundary.  What is outside the part is copied in pieces of its
// own width, or left alone in place.  The first pieces are on their way while the
// table is made.
// 6,143 tokens x 48 heads x 128 in bf16: 27.0 us as halves, 27.9 as neighbouring pairs, 27.6 with 96 dims turning (151 MB,
// 22.6 us at the copy rate); 34,065 x 16 x 128 in fp32: 82.9 us, the rate of a copy; 4,093 x 16 x 80 with 20 dims turning,
// pieces of 4 bytes: 5.0 us (with copies of 4 bytes too 9.6).
// The table keeps (cos, sin) of pair i of every piece side by side, so that
// neighbouring threads read neighbouring words (no bank conflicts).
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kFormThreads = 256;
constexpr int kFormMaxTokens = 8;  // of a block

// n / d for n < 2^31 by a multiplication: m = ceil(2^(32 + shift) / d) - 2^32 with
// shift = ceil(log2 d).
struct Divisor {
    uint32_t d, m, shift;
};
Divisor divisor(uint32_t d) {
    Divisor r{d, 0, 0};
    while ((1ull << r.shift) < d) ++r.shift;
    r.m = static_cast<uint32_t>((((1ull << r.shift) - d) << 32) / d + 1);
    return r;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& d) { return (__umulhi(n, d.m) + n) >> d.shift; }

struct FormParams {
    RopeFormDev form;
    const void* x;
    void* out;
    int64_t x_stride, out_stride, pos_stride, n;
    const int32_t* pos;
    int heads, back;
    int tokens;                    // of a block
    int copy;                      // dims of a piece that is copied; 0: none is
    Divisor turned, turned_row;    // pieces of a head that turn (halves: pairs of pieces), and of a token
    Divisor copied, copied_row;    // pieces of a head that are copied, and of a token
};

struct __align__(16) Piece32 {
    uint4 x, y;
};
template <int BYTES>
struct Piece;
template <>
struct Piece<32> { using type = Piece32; };
template <>
struct Piece<16> { using type = uint4; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<2> { using type = uint16_t; };

template <typename T, int V>
__device__ __forceinline__ void open_piece(const typename Piece<V * sizeof(T)>::type& w, float (&x)[V]) {
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = static_cast<float>(e[i]);
}
template <typename T, int V>
__device__ __forceinline__ typename Piece<V * sizeof(T)>::type close_piece(const float (&x)[V]) {
    typename Piece<V * sizeof(T)>::type w;
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = static_cast<T>(x[i]);
    return w;
}

// What does not turn, in pieces of type W: those in front of the part that turns, then those behind it.
template <typename T, typename W>
__device__ __forceinline__ void copy_pieces(const FormParams& p, const T* x, T* out, int nt) {
    constexpr int kUnroll = 4, kDims = sizeof(W) / sizeof(T);
    const uint32_t total = static_cast<uint32_t>(nt) * p.copied_row.d;
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kFormThreads * kUnroll) {
        W w[kUnroll];
        T* to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t i = i0 + u * kFormThreads;
            if (i >= total) continue;
            const int t = static_cast<int>(divide(i, p.copied_row));
            const uint32_t in_row = i - t * p.copied_row.d, h = divide(in_row, p.copied);
            int d = static_cast<int>(in_row - h * p.copied.d) * kDims;
            if (d >= p.form.first) d += p.form.dims;
            const int e = static_cast<int>(h) * p.form.head_dim + d;
            w[u] = *reinterpret_cast<const W*>(x + t * p.x_stride + e);
            to[u] = out + t * p.out_stride + e;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i0 + u * kFormThreads < total) *reinterpret_cast<W*>(to[u]) = w[u];
    }
}

template <typename T, int V, bool HALVES>
__global__ void __launch_bounds__(kFormThreads) rope_form_kernel(const __grid_constant__ FormParams p) {
    using W = typename Piece<V * sizeof(T)>::type;
    constexpr int kUnroll = HALVES || V * sizeof(T) == 32 ? 2 : 4;
    constexpr int kPairs = HALVES ? V : V / 2;  // of an item
    __shared__ float2 table[kFormMaxTokens * RC_ROPE_MAX_HEAD_DIM / 2];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.n - t0));
    const T* x = static_cast<const T*>(p.x) + t0 * p.x_stride;
    T* out = static_cast<T*>(p.out) + t0 * p.out_stride;
    const int half = p.form.dims / 2, turned = static_cast<int>(p.turned.d);
    const uint32_t total = static_cast<uint32_t>(nt) * p.turned_row.d;

    // an item: token, first element, place among a head's items
    struct Item {
        int t, e, c;
    };
    Item it[kUnroll];
    W a[kUnroll], b[kUnroll];
    auto load_all = [&](uint32_t i0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint32_t i = i0 + u * kFormThreads;
            if (i >= total) continue;
            it[u].t = static_cast<int>(divide(i, p.turned_row));
            const uint32_t in_row = i - it[u].t * p.turned_row.d, h = divide(in_row, p.turned);
            it[u].c = static_cast<int>(in_row - h * p.turned.d);
            it[u].e = static_cast<int>(h) * p.form.head_dim + p.form.first + it[u].c * V;
            const T* from = x + it[u].t * p.x_stride + it[u].e;
            a[u] = *reinterpret_cast<const W*>(from);
            if (HALVES) b[u] = *reinterpret_cast<const W*>(from + half);
        }
    };
    load_all(threadIdx.x);

    {
        const uint64_t* turns = param_address(p.form.turns);
        const uint8_t* axis = param_address(p.form.axis);
        for (int i = threadIdx.x; i < nt * half; i += kFormThreads) {
            const int t = i / half, c = i - t * half;
            const float2 cs = turn_cos_sin(__ldg(p.pos + axis[c] * p.pos_stride + t0 + t), turns[c]);
            table[t * half + (c % kPairs) * turned + c / kPairs] =
                make_float2(p.form.gain * cs.x, (p.back ? -p.form.gain : p.form.gain) * cs.y);
        }
    }
    __syncthreads();
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kFormThreads * kUnroll) {
        if (i0 != threadIdx.x) load_all(i0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i0 + u * kFormThreads >= total) continue;
            T* to = out + it[u].t * p.out_stride + it[u].e;
            const float2* cs = table + it[u].t * half + it[u].c;
            float xa[V];
            open_piece<T, V>(a[u], xa);
            if (HALVES) {
                float xb[V];
                open_piece<T, V>(b[u], xb);
#pragma unroll
                for (int i = 0; i < V; ++i) rotate_pair(xa[i], xb[i], cs[i * turned].x, cs[i * turned].y, xa[i], xb[i]);
                *reinterpret_cast<W*>(to + half) = close_piece<T, V>(xb);
            } else {
#pragma unroll
                for (int i = 0; i < V / 2; ++i)
                    rotate_pair(xa[2 * i], xa[2 * i + 1], cs[i * turned].x, cs[i * turned].y, xa[2 * i], xa[2 * i + 1]);
            }
            *reinterpret_cast<W*>(to) = close_piece<T, V>(xa);
        }
    }
    switch (p.copy * static_cast<int>(sizeof(T))) {
        case 16: copy_pieces<T, uint4>(p, x, out, nt); break;
        case 8: copy_pieces<T, uint2>(p, x, out, nt); break;
        case 4: copy_pieces<T, uint32_t>(p, x, out, nt); break;
    }
}

template <typename T, int V, bool HALVES>
cudaError_t launch_v(FormParams& p, cudaStream_t s) {
    const uint32_t heads = static_cast<uint32_t>(p.heads), turned = static_cast<uint32_t>(p.form.dims / (HALVES ? 2 * V : V));
    p.turned = divisor(turned);
    p.turned_row = divisor(turned * heads);
    // copies go with the turn, unless the result lies where x does; 16 bytes at a time at most
    constexpr int kMost = 16 / sizeof(T);
    const int grain = p.form.first | (p.form.first + p.form.dims) | p.form.head_dim | kMost;  // (all even)
    p.copy = p.x == p.out || p.form.dims == p.form.head_dim ? 0 : grain & -grain;
    if (p.copy) {
        const uint32_t copied = static_cast<uint32_t>((p.form.head_dim - p.form.dims) / p.copy);
        p.copied = divisor(copied);
        p.copied_row = divisor(copied * heads);
    }
    // Tokens of a block: enough blocks to fill the card first, then up to 2,048 pieces of 16 bytes.
    const int64_t bytes = static_cast<int64_t>(p.heads) * p.form.head_dim * sizeof(T);
    p.tokens = 1;
    while (p.tokens < kFormMaxTokens && p.n / (2 * p.tokens) >= 152 * 4 && bytes * p.tokens < 8 * kFormThreads * 16) p.tokens *= 2;
    const int64_t grid = (p.n + p.tokens - 1) / p.tokens;
    rope_form_kernel<T, V, HALVES><<<static_cast<unsigned>(grid), kFormThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool HALVES>
cudaError_t launch_t(FormParams& p, cudaStream_t s) {
    // pieces on V's boundary: the part's start and its half (neighbours: its length)
    const int grain = p.form.first | (HALVES ? p.form.dims / 2 : p.form.dims);
    if constexpr (!HALVES)
        if (grain % (32 / sizeof(T)) == 0) return launch_v<T, 32 / sizeof(T), HALVES>(p, s);
    if constexpr (sizeof(T) == 2)
        if (grain % 8 == 0) return launch_v<T, 8, HALVES>(p, s);
    if (grain % 4 == 0) return launch_v<T, 4, HALVES>(p, s);
    if (grain % 2 == 0) return launch_v<T, 2, HALVES>(p, s);
    if constexpr (HALVES)
        return launch_v<T, 1, HALVES>(p, s);
    else
        return cudaErrorInvalidValue;  // (both are even)
}

}  // namespace

cudaError_t launch_rope_form(const RopeFormParams& q, int dtype, cudaStream_t s) {
    FormParams p{};
    p.form = q.form;
    p.x = q.x;
    p.out = q.out;
    p.x_stride = q.x_stride;
    p.out_stride = q.out_stride;
    p.pos_stride = q.pos_stride;
    p.n = q.n;
    p.pos = q.pos;
    p.heads = q.heads;
    p.back = q.back;
    const bool halves = p.form.layout == RC_ROPE_HALVES;
    if (dtype == RC_BF16) return halves ? launch_t<__nv_bfloat16, true>(p, s) : launch_t<__nv_bfloat16, false>(p, s);
    return halves ? launch_t<float, true>(p, s) : launch_t<float, false>(p, s);
}

}  // namespace rc
