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

    // A tile's words and scales.  Loads are what a compute unit runs out of (one
    // in about 25 cycles, whatever its width), so four scales of a row of W come
    // in one load, one to each 16 lanes, and are handed around in registers:
    // scale (j, g) is number GROUPS j + g.
    static constexpr int COUNT = NT * GROUPS, EACH = COUNT < 4 ? COUNT : 4, LOADS = COUNT / EACH;
    struct Weights {
        u32x4 words[NT];
        S raw[LOADS];
        float scale[COUNT];
        __device__ void load(const u32x4* const* tiles, const S* const* scales, uint32_t tk, uint32_t lane) {
#pragma unroll
            for (int j = 0; j < NT; ++j) words[j] = __builtin_nontemporal_load(tiles[j] + (uint64_t)tk * 64 + lane);
#pragma unroll
            for (int q = 0; q < LOADS; ++q) raw[q] = scales[q][(uint64_t)tk * (GROUPS * 16)];
        }
        __device__ void spread() {
#pragma unroll
            for (int q = 0; q < LOADS; ++q) {
                const uint32_t v = __float_as_uint((float)raw[q] * O::SCALE);
                if constexpr (EACH == 1) {
                    scale[q] = __uint_as_float(v);
                } else {
                    // rows of 16 lanes 0 1 2 3 -> 0 0 2 2 and 1 1 3 3 -> each everywhere
                    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
                    if constexpr (EACH == 2) {
                        scale[2 * q] = __uint_as_float(p[0]);
                        scale[2 * q + 1] = __uint_as_float(p[1]);
                    } else {
                        const auto a = __builtin_amdgcn_permlane32_swap(p[0], p[0], false, false);
                        const auto b = __builtin_amdgcn_permlane32_swap(p[1], p[1], false, false);
                        scale[4 * q] = __uint_as_float(a[0]);
                        scale[4 * q + 1] = __uint_as_float(b[0]);
                        scale[4 * q + 2] = __uint_as_float(a[1]);
                        scale[4 * q + 3] = __uint_as_float(b[1]);
                    }
                }
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
                        finish(i, j, O::mul(x, q, Acc{0, 0, 0, 0}), w.scale[j * GROUPS + 2 * H + d]);
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
                    const float s = w.scale[j * GROUPS + H * GROUPS / 2];
#pragma unroll
                    for (int i = 0; i < MT; ++i) finish(i, j, acc[i][j], s);
                }
            }
        } else {
            constexpr int N = WORDS == 1 ? 1 : 2;   // words of a group in this half
#pragma unroll
            for (int g = 0; g < 2 / N; ++g)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    u32x4 q[N];
#pragma unroll
                    for (int d = 0; d < N; ++d) q[d] = O::weights(w.words[j][2 * H + g * N + d]);
                    const float s = w.scale[j * GROUPS + (WORDS == 4 ? 0 : H * GROUPS / 2 + g)];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        Acc v = WORDS == 4 && H == 1 ? acc[i][j] : Acc{0, 0, 0, 0};
#pragma unroll
                        for (int d = 0; d < N; ++d) v = O::mul(h.x[i][g * N + d], q[d], v);
                        if (WORDS == 4 && H == 0)
                            acc[i][j] = v;
                        else
                            finish(i, j, v, s);
                    }
                }
        }
    }
};

// A wave's tiles, every `waves`-th from `first` to `end`: fetch(d, tile) for DEPTH
// of them ahead of add(d).  Past its last tile a wave fetches that one again.
template <int DEPTH, typename Fetch, typename Add>
__device__ __forceinline__ void run(uint32_t first, uint32_t waves, uint32_t end, Fetch fetch, Add add) {
    if (first >= end) return;
    const uint32_t mine = (end - first + waves - 1) / waves;
    auto tile = [&](uint32_t t) { return first + (t < mine ? t : mine - 1) * waves; };
    uint32_t t = 0;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) fetch(d, tile(d));
    for (; t + DEPTH < mine; t += DEPTH)
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            add(d);
            __builtin_amdgcn_sched_barrier(0);   // mixed, the tiles' work runs out of registers
            fetch(d, tile(t + DEPTH + d));
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (t + d < mine) {
            add(d);
            __builtin_amdgcn_sched_barrier(0);
        }
}

// Waves of a workgroup: as many as the registers leave room for.
constexpr int few_waves(int mt, int nt) { return mt * nt == 1 ? 16 : 8; }
// Tiles that a wave has on their way or in registers.
constexpr int few_depth(int mt, int nt) { return nt == 4 ? 2 : mt == 2 ? 5 - nt : nt == 1 ? 4 : 3; }

// Tokens of their rows' tile, few enough that the 16 lanes of an instruction's
// tokens load several words' columns at once: lane 16 c + r takes eight columns
// of token r % ROWS; for word d they are then moved to lanes r < ROWS.
template <typename X, int ROWS>
struct InRows {
    typedef Operand<X> O;
    typedef typename O::A A;
    static constexpr int LOADS = ROWS / 4, PER = 16 / ROWS;   // words a load
    A v[LOADS];
    static __device__ uint32_t column(int i, uint32_t r, uint32_t c) { return 32 * (i * PER + r / ROWS) + 8 * c; }
    __device__ void load(const X* tile, uint32_t r, uint32_t c) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) v[i] = load_eight(tile, column(i, r, c));
    }
    __device__ void load(const X* tile, uint32_t r, uint32_t c, uint32_t left) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) v[i] = load_eight(tile, column(i, r, c), left);
    }
    __device__ void order() {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) v[i] = O::order(v[i]);
    }
    template <int D>
    __device__ A word() const {
        A a = v[D / PER];
        constexpr int FROM = D % PER * ROWS;   // lane r takes lane r + FROM of its sixteen
        if constexpr (FROM > 0) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(A) / 4); ++i)
                a[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a[i], 0x120 + 16 - FROM, 0xf, 0xf, true);
        }
        return a;
    }
    template <int H, typename Half>
    __device__ void half(Half& h) const {
        if constexpr (sizeof(X) == 1) {
            h.x[0][0] = Tokens<X>::join(word<2 * H>(), word<2 * H + 1>());
        } else {
            h.x[0][0] = word<2 * H>();
            h.x[0][1] = word<2 * H + 1>();
        }
    }
};

// One workgroup: 16 NT rows of W times 16 MT tokens, laid out (ROWS = 0), or
// times ROWS tokens in their rows.  Its waves share the columns out, tile by
// tile, each with the next tiles' loads in flight while it works on one, and
// add their sums up in LDS in a fixed order.  (64 tokens' tiles are too large
// for that: their words are one tile ahead, tokens half of one.)  Where there are
// few rows of W and many columns, several workgroups share the columns of a block
// (blockIdx.z); add_parts_kernel adds their sums up.
//
// One token: bound by HBM where W is large (28672 x 8192: int8 25 us, 4.8 TB/s; bf16
// 28 us, as making operands of the words that come last is not hidden; W is read
// once and does not stay in the cache) and by latency where it is not (4096 x 4096
// int8 4.2 us).  More tokens: by loads, of which a tile takes PIECES MT + NT + 1 or
// more (8192 x 8192: 32 tokens int8 11 us, bf16 14; 64 tokens int8 14, bf16 18).
// One token with three tiles in flight, 16 waves or two tiles of rows instead of
// four: 31, 33 and 29 us where this took 29.
template <typename X, typename S, int GROUP, int MT, int NT, int ROWS>
__global__ __launch_bounds__(64 * few_waves(MT, NT)) void matvec_w4_kernel(MatvecArgs a) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    typedef Sums<X, S, GROUP, MT, NT> Su;
    static_assert(ROWS == 0 || MT == 1, "tokens in rows: 16 at most");
    constexpr int COLS = 16 * NT, PITCH = COLS + 4;   // outputs of a token; + 4: rows on other banks
    constexpr int TOKENS = ROWS ? ROWS : 16 * MT;
    __shared__ float part[few_waves(MT, NT)][TOKENS][PITCH];
    const uint32_t waves = blockDim.x >> 6, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint32_t n0 = blockIdx.x * NT, mt0 = blockIdx.y * MT;
    const uint32_t share = (a.kt + a.splits - 1) / a.splits, from = blockIdx.z * share;
    const uint32_t until = from + share < a.kt ? from + share : a.kt;   // tiles of this workgroup (none: zeros)
    // tiles past the last repeat it: their sums are not stored
    auto tile_row = [&](uint32_t j) -> uint64_t { return n0 + j < a.nt ? n0 + j : a.nt - 1; };
    const u32x4* tiles[NT];
    const S* scales[Su::LOADS];
#pragma unroll
    for (int j = 0; j < NT; ++j) tiles[j] = a.tiles + tile_row(j) * a.kt * 64;
#pragma unroll
    for (int q = 0; q < Su::LOADS; ++q) {
        const uint32_t i = q * Su::EACH + c % Su::EACH;   // this lane's scale
        scales[q] = reinterpret_cast<const S*>(a.scales) + tile_row(i / Su::GROUPS) * a.kt * (Su::GROUPS * 16) +
                    i % Su::GROUPS * 16 + r;
    }
    Su sums;
    sums.clear();
    if constexpr (ROWS > 0) {
        constexpr int DEPTH = few_depth(MT, NT);
        typedef InRows<X, ROWS> Rows;
        const X* row = reinterpret_cast<const X*>(a.x) + (r % ROWS < a.m ? r % ROWS : a.m - 1) * a.x_stride;
        const uint32_t whole = (uint32_t)(a.k / TILE_COLS);
        typename Su::Weights w[DEPTH];
        Rows x[DEPTH];
        auto add = [&](typename Su::Weights& ww, Rows& xx) {
            typename Su::Half h;
            ww.spread();
            xx.order();
            xx.template half<0>(h);
            sums.template add<0>(ww, h);
            xx.template half<1>(h);
            sums.template add<1>(ww, h);
        };
        run<DEPTH>(
            from + wave, waves, until < whole ? until : whole,
            [&](int d, uint32_t tk) {
                x[d].load(row + (uint64_t)tk * TILE_COLS, r, c);
                w[d].load(tiles, scales, tk, lane);
            },
            [&](int d) { add(w[d], x[d]); });
        if (whole < until && from <= whole && wave == (whole - from) % waves) {   // the columns that do not fill a tile
            x[0].load(row + (uint64_t)whole * TILE_COLS, r, c, (uint32_t)(a.k % TILE_COLS));
            w[0].load(tiles, scales, whole, lane);
            add(w[0], x[0]);
        }
    } else {
        const u32x4* laid[MT];
        const uint32_t last = (uint32_t)((a.m - 1) / 16);   // tokens past the last sixteen repeat them
#pragma unroll
        for (int i = 0; i < MT; ++i)
            laid[i] = laid_tokens(a) + (uint64_t)(mt0 + i < last ? mt0 + i : last) * a.kt * (T::PIECES * 64);
        auto load = [&](typename Su::Half& h, uint32_t tk, uint32_t half) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int p = 0; p < Su::HALF; ++p)
                    h.x[i][p] = (laid[i] + ((uint64_t)tk * T::PIECES + half * Su::HALF + p) * 64)[lane];
        };
        if constexpr (MT <= 2) {
            constexpr int DEPTH = few_depth(MT, NT);
            typename Su::Weights w[DEPTH];
            typename Su::Half h[DEPTH][2];
            run<DEPTH>(
                from + wave, waves, until,
                [&](int d, uint32_t tk) {
                    load(h[d][0], tk, 0);
                    load(h[d][1], tk, 1);
                    w[d].load(tiles, scales, tk, lane);
                },
                [&](int d) {
                    w[d].spread();
                    sums.template add<0>(w[d], h[d][0]);
                    sums.template add<1>(w[d], h[d][1]);
                });
        } else {
            typename Su::Weights w0, w1;
            typename Su::Half h0, h1;
            uint32_t tk = from + wave;
            if (tk < until) {
                load(h0, tk, 0);
                w0.load(tiles, scales, tk, lane);
            }
            while (tk < until) {
                const uint32_t t1 = tk + waves, t2 = t1 + waves;
                load(h1, tk, 1);
                if (t1 < until) w1.load(tiles, scales, t1, lane);
                w0.spread();
                sums.template add<0>(w0, h0);
                if (t1 < until) load(h0, t1, 0);
                sums.template add<1>(w0, h1);
                if (t1 >= until) break;
                load(h1, t1, 1);
                if (t2 < until) w0.load(tiles, scales, t2, lane);
                w1.spread();
                sums.template add<0>(w1, h0);
                if (t2 < until) load(h0, t2, 0);
                sums.template add<1>(w1, h1);
                tk = t2;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (16 * i + 4 * c + e < TOKENS) part[wave][16 * i + 4 * c + e][16 * j + r] = sums.sum[i][j][e];
    lds_barrier();
    // the lanes of all waves share the outputs out, four neighbours each
    for (uint32_t at = threadIdx.x; at < TOKENS * COLS / 4; at += blockDim.x) {
        const uint32_t t = at / (COLS / 4), n = at % (COLS / 4) * 4;
        const uint64_t token = (uint64_t)mt0 * 16 + t, col = (uint64_t)n0 * 16 + n;
        if (token >= a.m || col >= a.n) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(&part[0][t][n]);
        for (uint32_t w = 1; w < waves; ++w) v += *reinterpret_cast<const f32x4*>(&part[w][t][n]);
        v *= O::FACTOR;
        if (a.splits > 1)
            *reinterpret_cast<f32x4*>(a.parts + (blockIdx.z * a.m + token) * (16 * (uint64_t)a.nt) + col) = v;
        else
            store_y(a, token, col, v);
    }
}

// The shares' sums, four outputs a lane, in the order of the columns.
__global__ __launch_bounds__(64) void add_parts_kernel(MatvecArgs a) {
    const uint64_t at = (uint64_t)blockIdx.x * 64 + threadIdx.x, row = 4 * (uint64_t)a.nt;   // fours of a token
    if (at >= a.m * row) return;
    const uint64_t token = at / row, col = at % row * 4;
    if (col >= a.n) return;
    f32x4 v = {0, 0, 0, 0};
    for (uint32_t z = 0; z < a.splits; ++z)
        v += *reinterpret_cast<const f32x4*>(a.parts + ((z * a.m + token) * row * 4 + col));
    store_y(a, token, col, v);
}

template <typename X, typename S, int GROUP, int MT, int NT, int ROWS>
int launch_few(const MatvecArgs& a, hipStream_t s) {
    // No more waves than have DEPTH tiles each, but four: what a wave asks for past
    // its last tile costs loads, a wave more only a share of the last sums.
    uint32_t waves = few_waves(MT, NT);
    while (waves > 4 && waves * few_depth(MT, NT) > tiles_of(a.kt, a.splits)) waves /= 2;
    matvec_w4_kernel<X, S, GROUP, MT, NT, ROWS>
        <<<dim3((uint32_t)tiles_of(a.nt, NT), (uint32_t)tiles_of(a.m, 16 * MT), a.splits), waves * 64, 0, s>>>(a);
    if (a.splits > 1)
        add_parts_kernel<<<dim3((uint32_t)tiles_of(a.m * a.nt, 16)), 64, 0, s>>>(a);
    return launched();
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, bool rows, hipStream_t s) {
    // More rows of W for a wave spare loads of x, fewer make more workgroups:
    // as many as leave one workgroup per compute unit.
    const uint32_t cus = (uint32_t)device_cu_count();
    auto go = [&](auto mt, auto in_rows) -> int {
        constexpr int MT = decltype(mt)::value, ROWS = decltype(in_rows)::value;
        const uint64_t blocks = a.nt * tiles_of(a.m, 16 * MT);
        if constexpr (MT < 4) {
            if (blocks >= 4 * cus) return launch_few<X, S, GROUP, MT, 4, ROWS>(a, s);
        }
        if (blocks >= 2 * cus) return launch_few<X, S, GROUP, MT, 2, ROWS>(a, s);
        return launch_few<X, S, GROUP, MT, 1, ROWS>(a, s);
    };
    typedef std::integral_constant<int, 0> Laid;
    typedef std::integral_constant<int, 1> One;
    if (rows && a.m <= 4) return go(One(), std::integral_constant<int, 4>());
    if (rows && a.m <= 8) return go(One(), std::integral_constant<int, 8>());
    if (rows) return go(One(), std::integral_constant<int, 16>());
    if (a.m <= 16) return go(One(), Laid());
    if (a.m <= 32) return go(std::integral_constant<int, 2>(), Laid());
    return go(std::integral_constant<int, 4>(), Laid());
}

template <typename X>
int launch_as(const MatvecArgs& a, bool rows, int scale_type, uint32_t group, hipStream_t s) {
    auto go = [&](auto scale) -> int {
        typedef decltype(scale) S;
        if (group == 32) return launch_group<X, S, 32>(a, rows, s);
        if (group == 64) return launch_group<X, S, 64>(a, rows, s);
        return launch_group<X, S, 128>(a, rows, s);
    };
    return scale_type == LECB_BF16 ? go(__bf16()) : go(float());
}

// Whether tokens are read from their rows, without a launch to lay them out
// first (2.7 us, and as much of the host): always up to four, and up to 16 where
// rows are short; up to 16 too where their loads are aligned and, above eight, rows
// not too long.  In rows and laid out, us, in a graph: 5 x 1003 x 1111 bf16 5.2 and
// 6.3; 8192 x 8192 bf16, 8 tokens 10.5 and 14.2, 16 tokens 13.8 and 14.3; 8 tokens
// of 8191 columns 19.3 and 13.7; 1000 x 28672, 16 tokens, int8 14.2 and 13.2, bf16
// 14.9 and 15.3, of 28001 columns 28.0 and 15.4.  Both give the same bits: the same
// instructions on the same operands, in the same order.
bool in_rows(const MatvecArgs& a, uint64_t bytes) {
    if (a.m <= 4 || (a.m <= 16 && a.kt <= 16)) return true;
    const bool aligned = (reinterpret_cast<uintptr_t>(a.x) | a.x_stride * bytes) % (8 * bytes) == 0;
    return aligned && (a.m <= 8 || (a.m <= 16 && a.kt <= 64));
}

// Shares of the columns over workgroups: where the blocks of outputs (16 rows, up
// to 64 tokens) leave half of the compute units or more idle and every share
// keeps 32 tiles; up to four tokens, whose blocks are sooner done, from 128 tiles
// on.  The sums' launch takes 2.5 us.  1000 x 28672 bf16 without and with shares, us,
// in a graph: 1 token 12.2 and 9.5, 16 tokens 25.0 and 15.3, 64 tokens 56 and 25.
uint64_t splits_of(uint64_t m, uint64_t nt, uint64_t kt) {
    const uint64_t blocks = nt * tiles_of(m, m <= 16 ? 16 : m <= 32 ? 32 : 64);
    const uint64_t idle = (uint64_t)device_cu_count() / blocks, most = kt / (m <= 4 ? 64 : 32);
    const uint64_t s = idle < most ? idle : most;
    return s < 2 ? 1 : s < 8 ? s : 8;
}
uint64_t parts_bytes(uint64_t m, uint64_t nt, uint64_t kt) {
    const uint64_t s = splits_of(m, nt, kt);
    return s > 1 ? s * m * nt * 64 : 0;
}

// Whether the form for many tokens takes it.  A round of its workgroups (64 x 256
// outputs a compute unit) takes about 8/3 as long as one here (64 x 32):
// 8192 x 8192 bf16, 65 to 128 tokens, 36 to 40 us here and 62 there; 300 tokens, 92
// and 63; 28672 x 4096, 48 tokens, 42 and 37; 1024 x 8192, 512 tokens, 25 and 62.
bool many(const MatvecArgs& a) {
    if (a.m <= 32 || a.kt >= MM_TILES) return false;
    const uint64_t cus = (uint64_t)device_cu_count();
    const uint64_t rounds = (tiles_of(a.m, 64) * tiles_of(a.nt, 2) + cus - 1) / cus;
    return 3 * rounds > 2 * matmul_w4_turns(a);
}

// Asked for whatever the tokens' addresses are; 9 to 16 tokens of short rows are
// asked for it too, though they go by in_rows.
uint64_t laying_bytes(uint64_t m, uint64_t kt) {
    return m <= 4 || (m <= 8 && kt <= 16) ? 0 : laid_bytes(m, kt);
}
uint64_t bytes_of(uint64_t m, uint64_t n, uint64_t k) {
    const uint64_t kt = tiles_of(k, TILE_COLS);
    return m && n ? laying_bytes(m, kt) + parts_bytes(m, tiles_of(n, TILE_ROWS), kt) : 0;
}

// What one pass of launches takes; more tokens and rows go by several passes, one
// after another with the same workspace.  A grid has fewer than 2^32 lanes and
// 65536 workgroups along y: 64 tokens a workgroup of few tokens; of many, 512 lanes
// for 64 tokens x 16 tiles of rows or more; of laying out, 256 lanes for 16 tokens
// x one tile of columns or more (up to LAY_ACROSS, as launch_lay_tokens has it).
struct Pass {
    uint64_t tokens, rows;
};
Pass pass_of(uint64_t n, uint64_t k) {
    constexpr uint64_t ROW_TILES = 1u << 22;
    const uint64_t nt = tiles_of(n, TILE_ROWS), kt = tiles_of(k, TILE_COLS);
    const uint64_t products = (1u << 22) / tiles_of(nt < ROW_TILES ? nt : ROW_TILES, 16);
    const uint64_t laying = LAY_ACROSS / (kt < LAY_ACROSS ? kt : LAY_ACROSS);
    const uint64_t blocks = products < laying ? products : laying;
    return {LAID_TOKENS * (blocks < 65535 ? blocks : 65535), ROW_TILES * TILE_ROWS};
}

int launch_pass(const MatvecW4& m, hipStream_t s) {
    const uint64_t nt = tiles_of(m.n, TILE_ROWS), kt = tiles_of(m.k, TILE_COLS);
    const MatvecArgs a{m.x, m.xscale, reinterpret_cast<const u32x4*>(m.tiles), m.scales, m.y, m.ws, m.x_stride,
                       m.y_stride, m.n, m.k, m.m, (uint32_t)nt, (uint32_t)kt, m.xscale_stride, m.y_type,
                       (uint32_t)splits_of(m.m, nt, kt),
                       reinterpret_cast<float*>(static_cast<char*>(m.ws) + laying_bytes(m.m, kt))};
    const bool rows = in_rows(a, elem_bytes(m.x_type));
    if (!rows) {
        const bool are_many = many(a);
        const int rc = launch_lay_tokens(a, m.x_type, are_many, s);
        if (rc) return rc;
        if (are_many) return launch_matmul_w4(a, m.x_type, m.scale_type, m.group, s);
    }
    switch (m.x_type) {
        case LECB_I8: return launch_as<int8_t>(a, rows, m.scale_type, m.group, s);
        case LECB_BF16: return launch_as<__bf16>(a, rows, m.scale_type, m.group, s);
        default: return launch_as<_Float16>(a, rows, m.scale_type, m.group, s);
    }
}

}  // namespace

uint64_t matvec_w4_workspace(uint64_t m, uint64_t n, uint64_t k) {
    const Pass p = pass_of(n, k);
    if (m <= p.tokens && n <= p.rows) return bytes_of(m, n, k);
    uint64_t most = 0;
    for (const uint64_t tokens : {m < p.tokens ? m : p.tokens, m % p.tokens})
        for (const uint64_t rows : {n < p.rows ? n : p.rows, n % p.rows}) {
            const uint64_t b = bytes_of(tokens, rows, k);
            most = b > most ? b : most;
        }
    return most;
}

int launch_matvec_w4(const MatvecW4& m, void* stream) {
    const Pass p = pass_of(m.n, m.k);
    const uint64_t kt = tiles_of(m.k, TILE_COLS), scales = TILE_COLS / m.group * TILE_ROWS * elem_bytes(m.scale_type);
    for (uint64_t token = 0; token < m.m; token += p.tokens)
        for (uint64_t row = 0; row < m.n; row += p.rows) {
            MatvecW4 one = m;
            one.m = m.m - token < p.tokens ? m.m - token : p.tokens;
            one.n = m.n - row < p.rows ? m.n - row : p.rows;
            one.x = static_cast<const char*>(m.x) + token * m.x_stride * elem_bytes(m.x_type);
            if (m.xscale) one.xscale = m.xscale + token * m.xscale_stride;
            one.tiles = m.tiles + row / TILE_ROWS * kt * TILE_BYTES;
            one.scales = static_cast<const char*>(m.scales) + row / TILE_ROWS * kt * scales;
            one.y = static_cast<char*>(m.y) + (token * m.y_stride + row) * elem_bytes(m.y_type);
            const int rc = launch_pass(one, reinterpret_cast<hipStream_t>(stream));
            if (rc) return rc;
        }
    return LECB_OK;
}

}  // namespace lecb
