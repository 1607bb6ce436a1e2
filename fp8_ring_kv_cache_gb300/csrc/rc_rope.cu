// rc_rope.cu -- rotary positions with several axes (rc_rope_axes): each
// dimension pair of a head turned by angle = position on the pair's axis x the
// pair's frequency, forward or back.
//
// Bound by memory: every value is read and written once, 16 bytes a thread
// (34,065 tokens x 16 heads x 128 in fp32: 82 us for 559 MB, the rate of a copy;
// 757 tokens x 48 heads x 128 in bf16: 4.9 us, half of it the launch).
// The angles depend on the token alone, so a block computes its tokens' (cos,
// sin) once into shared memory and all heads read them there.
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kRopeThreads = 256;

// One 16-byte piece of a row turned; cs: the (cos, sin) of its pairs.
__device__ __forceinline__ uint4 turn_piece(uint4 w, const float2* cs, float sign, __nv_bfloat16) {
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        rotate_pair(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xFFFF0000u), cs[i].x, sign * cs[i].y, a, b);
        r[i] = pack_bf16(a, b);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ uint4 turn_piece(uint4 w, const float2* cs, float sign, float) {
    float r[4];
    rotate_pair(__uint_as_float(w.x), __uint_as_float(w.y), cs[0].x, sign * cs[0].y, r[0], r[1]);
    rotate_pair(__uint_as_float(w.z), __uint_as_float(w.w), cs[1].x, sign * cs[1].y, r[2], r[3]);
    return make_uint4(__float_as_uint(r[0]), __float_as_uint(r[1]), __float_as_uint(r[2]), __float_as_uint(r[3]));
}

// A block takes `tb` tokens (at most kRopeMaxTokens), all heads.
constexpr int kRopeMaxTokens = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(const __grid_constant__ RopeAxesParams p, int tb) {
    constexpr int kPairs = D / 2;
    constexpr int kValues = 16 / sizeof(T);  // of one piece
    constexpr int kUnroll = 4;
    __shared__ float2 table[kRopeMaxTokens][kPairs];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tb;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tb), p.n - t0));
    const uint64_t* turns = param_address(p.rope.turns);
    const uint8_t* axis = param_address(p.rope.axis);
    for (int i = threadIdx.x; i < nt * kPairs; i += kRopeThreads) {
        const int t = i / kPairs, c = i % kPairs;
        table[t][c] = turn_cos_sin(__ldg(p.pos + axis[c] * p.pos_stride + t0 + t), turns[c]);
    }
    __syncthreads();
    const float sign = p.inverse ? -1.f : 1.f;
    const int per_token = p.heads * (D / kValues);  // pieces
    const int total = nt * per_token;
    const T* x = static_cast<const T*>(p.x) + t0 * p.x_stride;
    T* out = static_cast<T*>(p.out) + t0 * p.out_stride;
    for (int i0 = threadIdx.x; i0 < total; i0 += kRopeThreads * kUnroll) {
        uint4 w[kUnroll];
        int t[kUnroll], e[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kRopeThreads;
            t[u] = i / per_token;
            e[u] = (i - t[u] * per_token) * kValues;
            if (i < total) w[u] = *reinterpret_cast<const uint4*>(x + t[u] * p.x_stride + e[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i0 + u * kRopeThreads < total)
                *reinterpret_cast<uint4*>(out + t[u] * p.out_stride + e[u]) =
                    turn_piece(w[u], &table[t[u]][(e[u] % D) / 2], sign, T());
    }
}

template <typename T>
cudaError_t launch_t(const RopeAxesParams& p, int D, cudaStream_t s) {
    const int64_t pieces = p.n * p.heads * D * static_cast<int64_t>(sizeof(T)) / 16;
    // Tokens of a block: enough blocks to fill the card first, then up to 2,048
    // pieces (34,065 tokens x 16 heads x 128 in fp32: 1,024 pieces 85.5 us, 2,048
    // 82.1 us, 4,096 84.2 us; 757 tokens x 48 heads in bf16: one token 5.0 us,
    // two 5.5, four 6.6)
    int tb = 1;
    while (tb < kRopeMaxTokens && p.n / (2 * tb) >= 152 * 4 && pieces / p.n * tb < 8 * kRopeThreads) tb *= 2;
    const int64_t grid = (p.n + tb - 1) / tb;
    if (D == 128)
        rope_axes_kernel<T, 128><<<static_cast<unsigned>(grid), kRopeThreads, 0, s>>>(p, tb);
    else
        rope_axes_kernel<T, 64><<<static_cast<unsigned>(grid), kRopeThreads, 0, s>>>(p, tb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesParams& p, int D, int dtype, cudaStream_t s) {
    return dtype == RC_BF16 ? launch_t<__nv_bfloat16>(p, D, s) : launch_t<float>(p, D, s);
}

}  // namespace rc
