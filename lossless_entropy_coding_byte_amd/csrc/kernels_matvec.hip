// Products of tokens with 4-bit weights: y = x W^T, W in tiles of 4-bit codes
// with group scales (lecb.h gives the layout).
#include "layers.hpp"

namespace lecb {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// A word's eight codes as the matrix instruction's operand, and eight entries
// of x in the order that matches it.  The order of k inside an instruction is
// free as long as both operands agree: codes come out as (j, j + 4) pairs for
// 16-bit operands, as even and odd columns for bytes.
//
// 16-bit x: 1.codes -- the code's four bits, its sign bit flipped, become the
// top mantissa bits of 16.0: the value 24 + q, two codes per shift and
// and-or.  The surplus 24 sum(x) is taken off by a product with the constant
// -24, whose result lies exactly where the sums lie.
// int8 x: a code's four bits are the upper half of a byte: 16 q, the factor is
// taken off at the end.
template <typename X>
struct Operand;

template <>
struct Operand<__bf16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr uint32_t SURPLUS = 0xC1C0C1C0u;   // -24, twice
    static __device__ A weights(uint32_t w) {
        w ^= 0x88888888u;
        constexpr uint32_t M = 0x00780078u, ONE = 0x41804180u;
        return {((w << 3) & M) | ONE, ((w >> 1) & M) | ONE, ((w >> 5) & M) | ONE, ((w >> 9) & M) | ONE};
    }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
template <>
struct Operand<_Float16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr uint32_t SURPLUS = 0xCE00CE00u;   // -24, twice
    static __device__ A weights(uint32_t w) {
        w ^= 0x88888888u;
        constexpr uint32_t M = 0x03C003C0u, ONE = 0x4C004C00u;
        return {((w << 6) & M) | ONE, ((w << 2) & M) | ONE, ((w >> 2) & M) | ONE, ((w >> 6) & M) | ONE};
    }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
};
__device__ inline u32x4 pair_order(u32x4 x) {   // entries 0..7 -> (0,4) (1,5) (2,6) (3,7)
    return {__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
            __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

template <>
struct Operand<int8_t> {
    typedef u32x2 A;
    typedef i32x4 Acc;
    static __device__ A weights(uint32_t w) { return {(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u}; }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0,
                                                     0, 0);
    }
};
__device__ inline u32x2 pair_order(u32x2 x) {   // entries 0..7 -> evens, odds
    return {__builtin_amdgcn_perm(x.y, x.x, 0x06040200u), __builtin_amdgcn_perm(x.y, x.x, 0x07050301u)};
}

// Eight entries of a row of x in operand order; the guarded form takes `count`
// of them (zeros past that) and is used where a row's last tile is partial.
template <typename X>
__device__ inline typename Operand<X>::A load_x8(const X* p) {
    typedef typename Operand<X>::A A;
    typedef A loose __attribute__((aligned(sizeof(X))));
    return pair_order(*reinterpret_cast<const loose*>(p));
}
template <typename X>
__device__ inline typename Operand<X>::A load_x8(const X* p, uint64_t count) {
    if (count >= 8) return load_x8(p);
    typename Operand<X>::A v{};
    constexpr int PER = 4 / sizeof(X), BITS = 8 * sizeof(X);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if ((uint64_t)i >= count) continue;
        const uint32_t e = sizeof(X) == 1 ? reinterpret_cast<const uint8_t*>(p)[i]
                                          : reinterpret_cast<const uint16_t*>(p)[i];
        v[i / PER] |= e << (BITS * (i % PER));
    }
    return pair_order(v);
}

struct MatvecArgs {
    const void* x;
    const float* xscale;
    const u32x4* tiles;
    const void* scales;
    void* y;
    uint64_t x_stride, y_stride, n, k, m;
    uint32_t kt;
    int xscale_stride, bf16_scales, y_type;
};

// One workgroup: 16 rows of W times 16 tokens.  Its four waves take every
// fourth tile of the row of tiles each and add their sums up in LDS.
template <typename X, int GROUP>
__global__ __launch_bounds__(256) void matvec_w4_kernel(MatvecArgs a) {
    typedef Operand<X> O;
    constexpr bool INT = sizeof(X) == 1;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint64_t tn = blockIdx.x, m0 = (uint64_t)blockIdx.y * 16;
    // operand columns past m repeat the last token: their sums are not stored
    const uint64_t token = m0 + r < a.m ? m0 + r : a.m - 1;
    const X* x = reinterpret_cast<const X*>(a.x) + token * a.x_stride;
    constexpr int WORDS = GROUP / 32, GROUPS = 4 / WORDS;
    f32x4 sum = {0, 0, 0, 0};
    for (uint32_t tk = wave; tk < a.kt; tk += 4) {
        const uint64_t tile = tn * a.kt + tk;
        const u32x4 words = a.tiles[tile * 64 + lane];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            typename O::Acc acc = {0, 0, 0, 0};
#pragma unroll
            for (int d = g * WORDS; d < (g + 1) * WORDS; ++d) {
                const uint64_t c0 = (uint64_t)tk * TILE_COLS + 32 * d + 8 * c;
                const auto b = load_x8<X>(c0 < a.k ? x + c0 : x, c0 < a.k ? a.k - c0 : 0);
                if constexpr (!INT) acc = O::mul(u32x4{O::SURPLUS, O::SURPLUS, O::SURPLUS, O::SURPLUS}, b, acc);
                acc = O::mul(O::weights(words[d]), b, acc);
            }
            const uint64_t at = (tile * GROUPS + g) * 16 + 4 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float s = a.bf16_scales ? (float)reinterpret_cast<const __bf16*>(a.scales)[at + i]
                                              : reinterpret_cast<const float*>(a.scales)[at + i];
                sum[i] = fmaf((float)acc[i], s, sum[i]);
            }
        }
    }
    __shared__ f32x4 part[4][64];
    part[wave][lane] = sum;
    __syncthreads();
    if (wave) return;
    sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    const uint64_t i = m0 + r;
    if (i >= a.m) return;
    if (INT) sum *= (a.xscale ? a.xscale[a.xscale_stride ? i : 0] : 1.0f) * 0.0625f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t j = tn * 16 + 4 * c + e;
        if (j >= a.n) continue;
        const uint64_t at = i * a.y_stride + j;
        if (a.y_type == LECB_F32)
            reinterpret_cast<float*>(a.y)[at] = sum[e];
        else if (a.y_type == LECB_BF16)
            reinterpret_cast<__bf16*>(a.y)[at] = (__bf16)sum[e];
        else
            reinterpret_cast<_Float16*>(a.y)[at] = (_Float16)sum[e];
    }
}

template <typename X>
int launch_as(const MatvecW4& a, hipStream_t s) {
    MatvecArgs b{a.x, a.xscale, reinterpret_cast<const u32x4*>(a.tiles), a.scales, a.y, a.x_stride, a.y_stride,
                 a.n, a.k, a.m, (uint32_t)tiles_of(a.k, TILE_COLS), a.xscale_stride, a.scale_type == LECB_BF16,
                 a.y_type};
    const uint64_t nt = tiles_of(a.n, TILE_ROWS), mt = tiles_of(a.m, 16);
    if (mt > 65535) return LECB_ERR_TOO_LARGE;
    const dim3 grid((uint32_t)nt, (uint32_t)mt);
    auto go = [&](auto group) {
        constexpr int G = decltype(group)::value;
        matvec_w4_kernel<X, G><<<grid, 256, 0, s>>>(b);
    };
    if (a.group == 32)
        go(std::integral_constant<int, 32>());
    else if (a.group == 64)
        go(std::integral_constant<int, 64>());
    else
        go(std::integral_constant<int, 128>());
    return launched();
}

}  // namespace

uint64_t matvec_w4_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

int launch_matvec_w4(const MatvecW4& a, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    switch (a.x_type) {
        case LECB_I8: return launch_as<int8_t>(a, s);
        case LECB_BF16: return launch_as<__bf16>(a, s);
        default: return launch_as<_Float16>(a, s);
    }
}

}  // namespace lecb
