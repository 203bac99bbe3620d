// Products of tokens with 4-bit weights: y = x W^T, W in tiles of 4-bit codes
// with group scales (lecb.h gives the layout).
//
// The weights are the matrix instructions' first operand (16 rows of W), the
// tokens the second (16 tokens), so a lane ends up with four neighbouring
// outputs of one token: y[token lane % 16][4 (lane / 16) .. + 3] of a tile.
#include "matvec.hpp"

namespace lecb {

namespace {

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
    if (a.m > 64) return launch_matmul_w4(b, a.x_type, a.scale_type, a.group, s);
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
