// Products of tokens with 4-bit weights: y = x W^T, W in tiles of 4-bit codes
// with group scales (lecb.h gives the layout).
//
// The weights are the matrix instructions' first operand (16 rows of W), the
// tokens the second (16 tokens), so a lane ends up with four neighbouring
// outputs of one token: y[token lane % 16][4 (lane / 16) .. + 3] of a tile.
#include "layers.hpp"

namespace lecb {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));

// A word's eight codes as the matrix instruction's operand, eight entries of x
// as the other, and their product.
//
// 16-bit x: the codes become q / 16, exactly: one conversion each (the even
// codes from the word, the odd ones from the word shifted by four, byte by
// byte) and one packing per pair.  int8 x: a code's four bits as the upper
// half of a byte, 16 q, even columns and odd columns in a register each; x is
// put into the same order.  FACTOR takes the sixteen off again, exactly.
template <typename X>
struct Operand;

__device__ inline void code_floats(uint32_t w, float* f) {   // f[i] = code i / 16
    uint32_t u = w >> 4;
    asm("" : "+v"(u));   // keeps one shift, so that every other conversion picks its byte itself
    f[0] = __builtin_amdgcn_cvt_off_f32_i4(w);
    f[1] = __builtin_amdgcn_cvt_off_f32_i4(u);
    f[2] = __builtin_amdgcn_cvt_off_f32_i4((w >> 8) & 255u);
    f[3] = __builtin_amdgcn_cvt_off_f32_i4((u >> 8) & 255u);
    f[4] = __builtin_amdgcn_cvt_off_f32_i4(w >> 16);
    f[5] = __builtin_amdgcn_cvt_off_f32_i4(u >> 16);
    f[6] = __builtin_amdgcn_cvt_off_f32_i4(w >> 24);
    f[7] = __builtin_amdgcn_cvt_off_f32_i4(u >> 24);
}

template <>
struct Operand<__bf16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float FACTOR = 16.0f;
    static __device__ A weights(uint32_t w) {
        float f[8];
        code_floats(w, f);
        A a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
        return a;
    }
    static __device__ A tokens(A x) { return x; }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
template <>
struct Operand<_Float16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float FACTOR = 16.0f;
    static __device__ A weights(uint32_t w) {
        float f[8];
        code_floats(w, f);
        A a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2 * i], f[2 * i + 1]));
        return a;
    }
    static __device__ A tokens(A x) { return x; }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
};
template <>
struct Operand<int8_t> {
    typedef u32x2 A;
    typedef i32x4 Acc;
    static constexpr float FACTOR = 0.0625f;
    static __device__ A weights(uint32_t w) { return {(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u}; }
    static __device__ A tokens(A x) {
        return {__builtin_amdgcn_perm(x.y, x.x, 0x06040200u), __builtin_amdgcn_perm(x.y, x.x, 0x07050301u)};
    }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0,
                                                     0, 0);
    }
    // two words at once: 64 columns an instruction, at twice the rate
    static __device__ Acc mul2(A a0, A a1, A b0, A b1, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{(int)a0.x, (int)a0.y, (int)a1.x, (int)a1.y},
                                                     i32x4{(int)b0.x, (int)b0.y, (int)b1.x, (int)b1.y}, c, 0, 0, 0);
    }
};

// Eight entries of a row of x; the guarded form takes `count` of them (zeros
// past that) and is used where a row's last tile is partial.
template <typename X>
__device__ inline typename Operand<X>::A load_x8(const X* p) {
    typedef typename Operand<X>::A A;
    typedef A loose __attribute__((aligned(sizeof(X))));
    return *reinterpret_cast<const loose*>(p);
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
    return v;
}

// Four neighbouring scales as loaded, and as numbers.
template <typename S>
struct Scales {
    typedef S raw __attribute__((ext_vector_type(4)));
    raw v;
    __device__ void load(const S* p) { v = *reinterpret_cast<const raw*>(p); }
    __device__ float operator[](int i) const { return (float)v[i]; }
};

// The last step of a sum: the token's factor, one rounding, four outputs.
__device__ inline void store_y(void* y, int type, uint64_t at, uint64_t left, f32x4 v) {
    if (left >= 4) {
        if (type == LECB_F32) {
            typedef f32x4 loose __attribute__((aligned(4)));
            *reinterpret_cast<loose*>(reinterpret_cast<float*>(y) + at) = v;
        } else if (type == LECB_BF16) {
            typedef bf16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<__bf16*>(y) + at) =
                bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
            typedef f16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<_Float16*>(y) + at) =
                f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if ((uint64_t)e >= left) continue;
        if (type == LECB_F32)
            reinterpret_cast<float*>(y)[at + e] = v[e];
        else if (type == LECB_BF16)
            reinterpret_cast<__bf16*>(y)[at + e] = (__bf16)v[e];
        else
            reinterpret_cast<_Float16*>(y)[at + e] = (_Float16)v[e];
    }
}

struct MatvecArgs {
    const void* x;
    const float* xscale;
    const u32x4* tiles;
    const void* scales;
    void* y;
    uint64_t x_stride, y_stride, n, k, m;
    uint32_t nt, kt;
    int xscale_stride, y_type;
};

// ---------------------------------------------------------------- few tokens

// What one wave needs for one column of tiles: the words of NT tiles (16 NT
// rows of W), their scales, and the tokens' entries of those 128 columns.
template <typename X, typename S, int GROUP, int MT, int NT>
struct Step {
    typedef Operand<X> O;
    static constexpr int GROUPS = 128 / GROUP, WORDS = GROUP / 32;
    u32x4 words[NT];
    Scales<S> scale[NT][GROUPS];
    typename O::A x[MT][4];

    __device__ void load_w(const u32x4* const* tiles, const S* const* scales, uint32_t tk) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            words[j] = __builtin_nontemporal_load(tiles[j] + (uint64_t)tk * 64);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) scale[j][g].load(scales[j] + ((uint64_t)tk * GROUPS + g) * 16);
        }
    }
    __device__ void load_x(const X* const* p, uint32_t tk) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) x[i][d] = load_x8(p[i] + (uint64_t)tk * TILE_COLS + 32 * d);
    }
    __device__ void load_x(const X* const* p, uint32_t tk, uint64_t left) {   // columns from p's on
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const uint64_t c = (uint64_t)tk * TILE_COLS + 32 * d;
                x[i][d] = load_x8(p[i] + (c < left ? c : 0), c < left ? left - c : 0);
            }
    }
    __device__ void add(f32x4 (&sum)[MT][NT]) const {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                typename O::A w[WORDS];
#pragma unroll
                for (int d = 0; d < WORDS; ++d) w[d] = O::weights(words[j][g * WORDS + d]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    typename O::Acc acc = {0, 0, 0, 0};
                    if constexpr (sizeof(X) == 1 && WORDS > 1) {
#pragma unroll
                        for (int d = 0; d < WORDS; d += 2)
                            acc = O::mul2(w[d], w[d + 1], O::tokens(x[i][g * WORDS + d]),
                                          O::tokens(x[i][g * WORDS + d + 1]), acc);
                    } else {
#pragma unroll
                        for (int d = 0; d < WORDS; ++d) acc = O::mul(w[d], O::tokens(x[i][g * WORDS + d]), acc);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][j][e] = fmaf((float)acc[e], scale[j][g][e], sum[i][j][e]);
                }
            }
    }
};

// Waves of a workgroup: as many as the registers of two steps leave room for.
constexpr int few_waves(int mt, int nt) { return mt * nt == 1 ? 16 : mt * nt <= 4 ? 8 : 4; }

// One workgroup: 16 NT rows of W times 16 MT tokens.  Its waves share the
// columns out, tile by tile, each with the next tile's loads in flight while
// it works on one, and add their sums up in LDS in a fixed order.
template <typename X, typename S, int GROUP, int MT, int NT>
__global__ __launch_bounds__(64 * few_waves(MT, NT)) void matvec_w4_kernel(MatvecArgs a) {
    typedef Operand<X> O;
    typedef Step<X, S, GROUP, MT, NT> St;
    extern __shared__ f32x4 part[];   // [wave][MT][NT][64]
    const uint32_t waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint32_t n0 = blockIdx.x * NT;
    const uint64_t m0 = (uint64_t)blockIdx.y * (16 * MT);
    const u32x4* tiles[NT];
    const S* scales[NT];
    const X* x[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {   // tiles past the last repeat it: their sums are not stored
        const uint64_t tn = n0 + j < a.nt ? n0 + j : a.nt - 1;
        tiles[j] = a.tiles + tn * a.kt * 64 + lane;
        scales[j] = reinterpret_cast<const S*>(a.scales) + tn * a.kt * (St::GROUPS * 16) + 4 * c;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {   // so do tokens past the last
        const uint64_t t = m0 + 16 * i + r < a.m ? m0 + 16 * i + r : a.m - 1;
        x[i] = reinterpret_cast<const X*>(a.x) + t * a.x_stride;
    }
    f32x4 sum[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) sum[i][j] = {0, 0, 0, 0};
    const uint32_t whole = (uint32_t)(a.k / TILE_COLS);
    {
        const X* xc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) xc[i] = x[i] + 8 * c;
        St s0, s1;
        uint32_t tk = wave;
        if (tk < whole) {
            s0.load_w(tiles, scales, tk);
            s0.load_x(xc, tk);
        }
        while (tk < whole) {
            const uint32_t t1 = tk + waves, t2 = t1 + waves;
            if (t1 < whole) {
                s1.load_w(tiles, scales, t1);
                s1.load_x(xc, t1);
            }
            s0.add(sum);
            if (t1 >= whole) break;
            if (t2 < whole) {
                s0.load_w(tiles, scales, t2);
                s0.load_x(xc, t2);
            }
            s1.add(sum);
            tk = t2;
        }
        if (whole < a.kt && wave == whole % waves) {   // the columns that do not fill a tile
            s0.load_w(tiles, scales, whole);
            s0.load_x(xc, whole, a.k > 8 * c ? a.k - 8 * c : 0);
            s0.add(sum);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[((wave * MT + i) * NT + j) * 64 + lane] = sum[i][j];
    __syncthreads();
    // the lanes of all waves share the outputs out
    for (uint32_t at = threadIdx.x; at < MT * NT * 64; at += blockDim.x) {
        f32x4 v = part[at];
        for (uint32_t w = 1; w < waves; ++w) v += part[w * (MT * NT * 64) + at];
        const uint32_t l = at & 63, j = at / 64 % NT, i = at / 64 / NT;
        const uint64_t t = m0 + 16 * i + (l & 15), col = (uint64_t)(n0 + j) * 16 + 4 * (l >> 4);
        if (t >= a.m || col >= a.n) continue;
        float f = O::FACTOR;
        if (a.xscale) f *= a.xscale[a.xscale_stride ? t : 0];
        store_y(a.y, a.y_type, t * a.y_stride + col, a.n - col, v * f);
    }
}

template <typename X, typename S, int GROUP, int MT, int NT>
int launch_few(const MatvecArgs& a, hipStream_t s) {
    const uint64_t mt = tiles_of(a.m, 16 * MT);
    if (mt > 65535) return LECB_ERR_TOO_LARGE;
    uint32_t waves = few_waves(MT, NT);   // no more than there are tiles to share
    while (waves > 1 && waves / 2 >= a.kt) waves /= 2;
    matvec_w4_kernel<X, S, GROUP, MT, NT>
        <<<dim3((uint32_t)tiles_of(a.nt, NT), (uint32_t)mt), waves * 64, waves * MT * NT * 1024, s>>>(a);
    return launched();
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, hipStream_t s) {
    // More rows of W for a wave spare loads of x, fewer make more workgroups:
    // as many as leave one workgroup per compute unit.
    const uint32_t cus = (uint32_t)device_cu_count();
    const int nt = a.nt >= 4 * cus ? 4 : a.nt >= 2 * cus ? 2 : 1;
    auto go = [&](auto mt) -> int {
        constexpr int MT = decltype(mt)::value;
        if constexpr (MT < 4) {
            if (nt == 4) return launch_few<X, S, GROUP, MT, 4>(a, s);
        }
        if (nt >= 2) return launch_few<X, S, GROUP, MT, 2>(a, s);
        return launch_few<X, S, GROUP, MT, 1>(a, s);
    };
    if (a.m <= 16) return go(std::integral_constant<int, 1>());
    if (a.m <= 32) return go(std::integral_constant<int, 2>());
    return go(std::integral_constant<int, 4>());
}

template <typename X>
int launch_as(const MatvecW4& a, hipStream_t s) {
    MatvecArgs b{a.x, a.xscale, reinterpret_cast<const u32x4*>(a.tiles), a.scales, a.y, a.x_stride, a.y_stride,
                 a.n, a.k, a.m, (uint32_t)tiles_of(a.n, TILE_ROWS), (uint32_t)tiles_of(a.k, TILE_COLS),
                 a.xscale_stride, a.y_type};
    auto go = [&](auto scale) -> int {
        typedef decltype(scale) S;
        if (a.group == 32) return launch_group<X, S, 32>(b, s);
        if (a.group == 64) return launch_group<X, S, 64>(b, s);
        return launch_group<X, S, 128>(b, s);
    };
    return a.scale_type == LECB_BF16 ? go(__bf16()) : go(float());
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
