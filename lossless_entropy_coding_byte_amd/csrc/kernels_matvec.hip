// Products of few tokens with 4-bit weights: y = x W^T, W in tiles of 4-bit
// codes with group scales (lecb.h gives the layout; kernels_matmul.hip holds
// the form for many tokens).
#include "matvec.hpp"

namespace lecb {

namespace {

// A wave's sums for 16 MT tokens and 16 NT rows of W, over its share of the
// columns.  An instruction's result is y[token 4 c + e][row r of W] in lane
// 16 c + r.  A tile's 128 columns are taken in halves, so that a group of 128
// has half of its sum in `acc` in between.
template <typename X, typename S, int GROUP, int MT, int NT>
struct Sums {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    typedef typename O::Acc Acc;
    static constexpr int GROUPS = 128 / GROUP, WORDS = GROUP / 32, HALF = T::PIECES / 2;
    f32x4 sum[MT][NT];
    Acc acc[MT][NT];

    struct Weights {   // a tile's words and scales
        u32x4 words[NT];
        S scale[NT][GROUPS];
        __device__ void load(const u32x4* const* tiles, const S* const* scales, uint32_t tk, uint32_t lane) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                words[j] = __builtin_nontemporal_load(tiles[j] + (uint64_t)tk * 64 + lane);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) scale[j][g] = (scales[j] + ((uint64_t)tk * GROUPS + g) * 16)[lane & 15];
            }
        }
    };
    struct Half {   // of a tile's columns, for all tokens
        u32x4 x[MT][HALF];
    };

    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) sum[i][j] = {0, 0, 0, 0};
    }
    __device__ void finish(int i, int j, const Acc& v, float s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[i][j][e] = fmaf((float)v[e], s, sum[i][j][e]);
    }
    template <int H>
    __device__ void add(const Weights& w, const Half& h) {
        if constexpr (sizeof(X) == 1 && WORDS == 1) {   // one unit, two groups
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    const u32x2 q = O::weights(w.words[j][2 * H + d]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const u32x2 x = d ? u32x2{h.x[i][0].z, h.x[i][0].w} : u32x2{h.x[i][0].x, h.x[i][0].y};
                        finish(i, j, O::mul(x, q, Acc{0, 0, 0, 0}), (float)w.scale[j][2 * H + d]);
                    }
                }
        } else if constexpr (sizeof(X) == 1) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const u32x2 q0 = O::weights(w.words[j][2 * H]), q1 = O::weights(w.words[j][2 * H + 1]);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i][j] = O::mul2(h.x[i][0], q0, q1, WORDS == 4 && H == 1 ? acc[i][j] : Acc{0, 0, 0, 0});
                if constexpr (WORDS == 2 || H == 1) {
                    const float s = (float)w.scale[j][H * GROUPS / 2];
#pragma unroll
                    for (int i = 0; i < MT; ++i) finish(i, j, acc[i][j], s);
                }
            }
        } else {
            constexpr int N = WORDS == 1 ? 1 : 2;   // words of a group in this half
#pragma unroll
            for (int g = 0; g < 2 / N; ++g) {
                const u32x4 over = {O::EXCESS, O::EXCESS, O::EXCESS, O::EXCESS};
                Acc none[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    none[i] = {0, 0, 0, 0};
#pragma unroll
                    for (int d = 0; d < N; ++d) none[i] = O::mul(h.x[i][g * N + d], over, none[i]);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    u32x4 q[N];
#pragma unroll
                    for (int d = 0; d < N; ++d) q[d] = O::weights(w.words[j][2 * H + g * N + d]);
                    const float s = (float)w.scale[j][WORDS == 4 ? 0 : H * GROUPS / 2 + g];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        Acc v = WORDS == 4 && H == 1 ? acc[i][j] : none[i];
#pragma unroll
                        for (int d = 0; d < N; ++d) v = O::mul(h.x[i][g * N + d], q[d], v);
                        if (WORDS == 4 && H == 1) v += none[i];
                        if (WORDS == 4 && H == 0)
                            acc[i][j] = v;
                        else
                            finish(i, j, v, s);
                    }
                }
            }
        }
    }
};

// Waves of a workgroup: as many as the registers leave room for.
constexpr int few_waves(int mt, int nt) { return mt * nt == 1 ? 16 : 8; }

// One workgroup: 16 NT rows of W times 16 MT tokens.  Its waves share the
// columns out, tile by tile, each with the next tile's words and the next
// half's tokens in flight while it works on one, and add their sums up in LDS
// in a fixed order.
template <typename X, typename S, int GROUP, int MT, int NT, bool LAID>
__global__ __launch_bounds__(64 * few_waves(MT, NT)) void matvec_w4_kernel(MatvecArgs a) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    typedef Sums<X, S, GROUP, MT, NT> Su;
    static_assert(LAID || MT == 1, "tokens in rows: 16 at most");
    constexpr int COLS = 16 * NT, PITCH = COLS + 4;   // outputs of a token; + 4: rows on other banks
    __shared__ float part[few_waves(MT, NT)][16 * MT][PITCH];
    const uint32_t waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint32_t n0 = blockIdx.x * NT, mt0 = blockIdx.y * MT;
    const u32x4* tiles[NT];
    const S* scales[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {   // tiles past the last repeat it: their sums are not stored
        const uint64_t tn = n0 + j < a.nt ? n0 + j : a.nt - 1;
        tiles[j] = a.tiles + tn * a.kt * 64;
        scales[j] = reinterpret_cast<const S*>(a.scales) + tn * a.kt * (Su::GROUPS * 16);
    }
    const u32x4* laid[MT];
    const X* row = nullptr;
    if constexpr (LAID) {
        const uint32_t last = (uint32_t)((a.m - 1) / 16);   // so do tokens past the last sixteen
#pragma unroll
        for (int i = 0; i < MT; ++i)
            laid[i] = laid_tokens(a) + (uint64_t)(mt0 + i < last ? mt0 + i : last) * a.kt * (T::PIECES * 64);
    } else {
        row = reinterpret_cast<const X*>(a.x) + (r < a.m ? r : a.m - 1) * a.x_stride;
    }
    Su sums;
    sums.clear();
    const uint32_t whole = LAID ? a.kt : (uint32_t)(a.k / TILE_COLS);
    auto load = [&](typename Su::Half& h, uint32_t tk, uint32_t half) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < Su::HALF; ++p) {
                if constexpr (LAID)
                    h.x[i][p] = (laid[i] + ((uint64_t)tk * T::PIECES + half * Su::HALF + p) * 64)[lane];
                else
                    h.x[i][p] = T::load(row + (uint64_t)tk * TILE_COLS, 4 * (half * Su::HALF + p) + c);
            }
    };
    auto ordered = [&](typename Su::Half h) {
        if constexpr (!LAID) {
#pragma unroll
            for (int p = 0; p < Su::HALF; ++p) h.x[0][p] = O::order(h.x[0][p]);
        }
        return h;
    };
    typename Su::Weights w0, w1;
    typename Su::Half h0, h1;
    uint32_t tk = wave;
    if (tk < whole) {
        load(h0, tk, 0);
        w0.load(tiles, scales, tk, lane);
    }
    while (tk < whole) {
        const uint32_t t1 = tk + waves, t2 = t1 + waves;
        load(h1, tk, 1);
        if (t1 < whole) w1.load(tiles, scales, t1, lane);
        sums.template add<0>(w0, ordered(h0));
        if (t1 < whole) load(h0, t1, 0);
        sums.template add<1>(w0, ordered(h1));
        if (t1 >= whole) break;
        load(h1, t1, 1);
        if (t2 < whole) w0.load(tiles, scales, t2, lane);
        sums.template add<0>(w1, ordered(h0));
        if (t2 < whole) load(h0, t2, 0);
        sums.template add<1>(w1, ordered(h1));
        tk = t2;
    }
    if constexpr (!LAID) {
        if (whole < a.kt && wave == whole % waves) {   // the columns that do not fill a tile
            const X* p = row + (uint64_t)whole * TILE_COLS;
            const uint32_t left = (uint32_t)(a.k % TILE_COLS);
            w0.load(tiles, scales, whole, lane);
#pragma unroll
            for (int i = 0; i < Su::HALF; ++i) {
                h0.x[0][i] = T::load(p, 4 * i + c, left);
                h1.x[0][i] = T::load(p, 4 * (Su::HALF + i) + c, left);
            }
            sums.template add<0>(w0, ordered(h0));
            sums.template add<1>(w0, ordered(h1));
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) part[wave][16 * i + 4 * c + e][16 * j + r] = sums.sum[i][j][e];
    lds_barrier();
    // the lanes of all waves share the outputs out, four neighbours each
    for (uint32_t at = threadIdx.x; at < MT * 16 * COLS / 4; at += blockDim.x) {
        const uint32_t t = at / (COLS / 4), n = at % (COLS / 4) * 4;
        const uint64_t token = (uint64_t)mt0 * 16 + t, col = (uint64_t)n0 * 16 + n;
        if (token >= a.m || col >= a.n) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(&part[0][t][n]);
        for (uint32_t w = 1; w < waves; ++w) v += *reinterpret_cast<const f32x4*>(&part[w][t][n]);
        store_y(a, token, col, v * O::FACTOR);
    }
}

template <typename X, typename S, int GROUP, int MT, int NT, bool LAID>
int launch_few(const MatvecArgs& a, hipStream_t s) {
    const uint64_t mt = tiles_of(a.m, 16 * MT);
    if (mt > 65535) return LECB_ERR_TOO_LARGE;
    uint32_t waves = few_waves(MT, NT);   // no more than there are tiles to share
    while (waves > 1 && waves / 2 >= a.kt) waves /= 2;
    matvec_w4_kernel<X, S, GROUP, MT, NT, LAID>
        <<<dim3((uint32_t)tiles_of(a.nt, NT), (uint32_t)mt), waves * 64, 0, s>>>(a);
    return launched();
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, hipStream_t s) {
    // More rows of W for a wave spare loads of x, fewer make more workgroups:
    // as many as leave one workgroup per compute unit.
    const uint32_t cus = (uint32_t)device_cu_count();
    auto go = [&](auto mt, auto laid) -> int {
        constexpr int MT = decltype(mt)::value;
        constexpr bool LAID = decltype(laid)::value;
        const uint64_t rows = a.nt * tiles_of(a.m, 16 * MT);
        if constexpr (MT < 4) {
            if (rows >= 4 * cus) return launch_few<X, S, GROUP, MT, 4, LAID>(a, s);
        }
        if (rows >= 2 * cus) return launch_few<X, S, GROUP, MT, 2, LAID>(a, s);
        return launch_few<X, S, GROUP, MT, 1, LAID>(a, s);
    };
    if (a.m <= FEW_IN_ROWS) return go(std::integral_constant<int, 1>(), std::false_type());
    if (a.m <= 16) return go(std::integral_constant<int, 1>(), std::true_type());
    if (a.m <= 32) return go(std::integral_constant<int, 2>(), std::true_type());
    return go(std::integral_constant<int, 4>(), std::true_type());
}

template <typename X>
int launch_as(const MatvecArgs& a, int scale_type, uint32_t group, hipStream_t s) {
    auto go = [&](auto scale) -> int {
        typedef decltype(scale) S;
        if (group == 32) return launch_group<X, S, 32>(a, s);
        if (group == 64) return launch_group<X, S, 64>(a, s);
        return launch_group<X, S, 128>(a, s);
    };
    return scale_type == LECB_BF16 ? go(__bf16()) : go(float());
}

bool many(const MatvecArgs& a) { return a.m > 64 && a.kt < MM_TILES; }

}  // namespace

uint64_t matvec_w4_workspace(uint64_t m, uint64_t, uint64_t k) {
    return m <= FEW_IN_ROWS ? 0 : laid_bytes(m, tiles_of(k, TILE_COLS));
}

int launch_matvec_w4(const MatvecW4& m, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const MatvecArgs a{m.x, m.xscale, reinterpret_cast<const u32x4*>(m.tiles), m.scales, m.y, m.ws, m.x_stride,
                       m.y_stride, m.n, m.k, m.m, (uint32_t)tiles_of(m.n, TILE_ROWS), (uint32_t)tiles_of(m.k, TILE_COLS),
                       m.xscale_stride, m.y_type};
    if (a.m > FEW_IN_ROWS) {
        const int rc = launch_lay_tokens(a, m.x_type, m.group, many(a), s);
        if (rc) return rc;
        if (many(a)) return launch_matmul_w4(a, m.x_type, m.scale_type, m.group, s);
    }
    switch (m.x_type) {
        case LECB_I8: return launch_as<int8_t>(a, m.scale_type, m.group, s);
        case LECB_BF16: return launch_as<__bf16>(a, m.scale_type, m.group, s);
        default: return launch_as<_Float16>(a, m.scale_type, m.group, s);
    }
}

}  // namespace lecb
