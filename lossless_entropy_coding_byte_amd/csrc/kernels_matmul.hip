// Products of many tokens with 4-bit weights: y = x W^T (lecb.h gives the
// layout of W, kernels_matvec.hip the form for few tokens).
//
// A workgroup takes 64 tokens and 64 WN rows of W; its eight waves are WN along
// the rows times 8 / WN along the columns.  A wave keeps 64 x 64 sums in
// registers: its words of W come from memory as the matrix instructions take
// them, are turned into numbers there and serve four instructions each; the
// tokens come through LDS, where the WN waves of one share of the columns put
// each tile of 128 columns once, in the order the instructions take them.
#include "matvec.hpp"

namespace lecb {

namespace {

// Waits for this wave's LDS accesses and then for the other waves.  Loads from
// memory stay in flight: only the lanes that asked for them read what they bring.
__device__ inline void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

constexpr int MM_WAVES = 8;
constexpr int MM_TOKENS = 64;
constexpr int MM_ROWS = 64;   // of W, a wave's

// A tile of tokens in LDS: 64 tokens x 128 columns as 16-byte units, each what
// one lane gives one matrix instruction (two in turn for bytes in groups of
// 32).  16-bit: unit u of a row holds columns 8 u ..; bytes: unit 4 p + c holds
// columns 64 p + 8 c .. and 64 p + 32 + 8 c ...  Lane (token r, c) of an
// instruction reads its unit at a place that the XOR spreads over the banks
// for the writes, where neighbouring lanes hold one token's units.
template <typename X>
struct Tokens {
    typedef Operand<X> O;
    static constexpr int UNITS = 8 * sizeof(X);   // per token
    static __device__ uint32_t place(uint32_t token, uint32_t unit) {
        return ((token >> 4) * UNITS + unit) * 16 + ((token & 15) ^ (16 / UNITS * unit));
    }
    static __device__ u32x4 load(const X* row, uint32_t unit) {
        if constexpr (sizeof(X) == 1) {
            const X* p = row + 64 * (unit >> 2) + 8 * (unit & 3);
            return join(load_x8(p), load_x8(p + 32));
        } else {
            return load_x8(row + 8 * unit);
        }
    }
    // zeros past `left` columns
    static __device__ u32x4 load(const X* row, uint32_t unit, uint32_t left) {
        if constexpr (sizeof(X) == 1) {
            const uint32_t c = 64 * (unit >> 2) + 8 * (unit & 3);
            return join(load_x8(row + (c < left ? c : 0), c < left ? left - c : 0),
                        load_x8(row + (c + 32 < left ? c + 32 : 0), c + 32 < left ? left - c - 32 : 0));
        } else {
            const uint32_t c = 8 * unit;
            return load_x8(row + (c < left ? c : 0), c < left ? left - c : 0);
        }
    }
    static __device__ u32x4 join(u32x2 a, u32x2 b) {
        a = Operand<int8_t>::tokens(a);
        b = Operand<int8_t>::tokens(b);
        return {a.x, a.y, b.x, b.y};
    }
};

template <typename X, typename S, int GROUP, int WN>
__global__ __launch_bounds__(64 * MM_WAVES) void matmul_w4_kernel(MatvecArgs a, uint32_t mblocks, uint32_t blocks) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    constexpr int WK = MM_WAVES / WN, GROUPS = 128 / GROUP, WORDS = GROUP / 32;
    constexpr int UNITS = MM_TOKENS * T::UNITS, P = UNITS / (64 * WN);   // units of a tile; a lane's share
    constexpr int COLS = MM_ROWS * WN, PITCH = COLS + 4;                 // outputs of a token; + 4: rows on other banks
    union Shared {
        u32x4 x[2][WK][UNITS];
        float y[WK][MM_TOKENS][PITCH];
    };
    __shared__ Shared sh;

    // Workgroups of one XCD (every eighth) take neighbouring rows of W, and the
    // blocks of tokens of the same rows are next to one another: what an XCD
    // reads of W it reads once.
    const uint32_t per = (blocks + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || id >= blocks) return;
    const uint32_t m0 = id % mblocks * MM_TOKENS, n0 = id / mblocks * (COLS / 16);   // token, tile of W
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave % WN, wk = wave / WN;
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;

    const u32x4* tiles[4];
    const S* scales[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // tiles past the last repeat it: their sums are not stored
        const uint64_t t = n0 + wn * 4 + j, tn = t < a.nt ? t : a.nt - 1;
        tiles[j] = a.tiles + tn * a.kt * 64;
        scales[j] = reinterpret_cast<const S*>(a.scales) + tn * a.kt * (GROUPS * 16);
    }
    const uint32_t share = wn * 64 + lane;   // of the tile's units
    const X* row[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {   // so do tokens past the last
        const uint64_t t = m0 + (p * (64 * WN) + share) / T::UNITS;
        row[p] = reinterpret_cast<const X*>(a.x) + (t < a.m ? t : a.m - 1) * a.x_stride;
    }
    const uint32_t whole = (uint32_t)(a.k / TILE_COLS), rest = (uint32_t)(a.k % TILE_COLS);

    u32x4 words[4], next_words[4], next_x[P];
    S scale[4][GROUPS];
    // A step's loads are in flight while the step before it is computed; the
    // columns that do not fill a tile are guarded loads and come with commit.
    auto fetch = [&](uint32_t tk) {
        if (tk < whole) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                next_x[p] = T::load(row[p] + (uint64_t)tk * TILE_COLS, (p * (64 * WN) + share) % T::UNITS);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) next_words[j] = (tiles[j] + (uint64_t)tk * 64)[lane];
    };
    auto commit = [&](uint32_t tk, uint32_t buffer) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            words[j] = next_words[j];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) scale[j][g] = (scales[j] + ((uint64_t)tk * GROUPS + g) * 16)[r];
        }
        u32x4* x = sh.x[buffer][wk];
        if (tk < whole) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const uint32_t u = p * (64 * WN) + share;
                x[T::place(u / T::UNITS, u % T::UNITS)] = next_x[p];
            }
        } else {
#pragma unroll 1
            for (uint32_t u = share; u < UNITS; u += 64 * WN) {
                const uint64_t t = m0 + u / T::UNITS;
                x[T::place(u / T::UNITS, u % T::UNITS)] =
                    T::load(reinterpret_cast<const X*>(a.x) + (t < a.m ? t : a.m - 1) * a.x_stride +
                                (uint64_t)tk * TILE_COLS, u % T::UNITS, rest);
            }
        }
    };

    f32x4 sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = {0, 0, 0, 0};

    auto compute = [&](uint32_t buffer) {
        const u32x4* x = sh.x[buffer][wk];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            typename O::Acc acc[4][4];
            if constexpr (sizeof(X) == 1 && WORDS > 1) {
#pragma unroll
                for (int d = 0; d < WORDS; d += 2) {
                    u32x4 xo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) xo[i] = x[T::place(16 * i + r, 4 * (g * WORDS / 2 + d / 2) + c)];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x2 w0 = O::weights(words[j][g * WORDS + d]), w1 = O::weights(words[j][g * WORDS + d + 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[i][j] = O::mul2({xo[i].x, xo[i].y}, {xo[i].z, xo[i].w}, w0, w1,
                                                d ? acc[i][j] : typename O::Acc{0, 0, 0, 0});
                    }
                }
            } else {
#pragma unroll
                for (int d = 0; d < WORDS; ++d) {
                    typename O::A xo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (sizeof(X) == 1) {   // one instruction takes half a unit
                            const u32x4 v = x[T::place(16 * i + r, 4 * (g / 2) + c)];
                            xo[i] = g & 1 ? u32x2{v.z, v.w} : u32x2{v.x, v.y};
                        } else {
                            xo[i] = x[T::place(16 * i + r, 4 * (g * WORDS + d) + c)];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const typename O::A w = O::weights(words[j][g * WORDS + d]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[i][j] = O::mul(xo[i], w, d ? acc[i][j] : typename O::Acc{0, 0, 0, 0});
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float s = (float)scale[j][g];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum[i][j][e] = fmaf((float)acc[i][j][e], s, sum[i][j][e]);
            }
        }
    };

    // Every wave takes the same number of steps; those past the last tile only wait.
    const uint32_t steps = (a.kt + WK - 1) / WK;
    if (wk < a.kt) {
        fetch(wk);
        commit(wk, 0);
    }
    for (uint32_t s = 0; s < steps; ++s) {
        const uint32_t tk = s * WK + wk;
        lds_barrier();   // this tile is there, and the last one is read
        if (tk + WK < a.kt) fetch(tk + WK);
        if (tk < a.kt) compute(s & 1);
        if (tk + WK < a.kt) commit(tk + WK, (s + 1) & 1);
    }

    // The columns' shares are added up in a fixed order, and a lane stores four
    // neighbouring outputs.
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sh.y[wk][16 * i + 4 * c + e][wn * MM_ROWS + 16 * j + r] = sum[i][j][e];
    lds_barrier();
    for (uint32_t at = threadIdx.x; at < MM_TOKENS * COLS / 4; at += 64 * MM_WAVES) {
        const uint32_t t = at / (COLS / 4), col = at % (COLS / 4) * 4;
        const uint64_t token = m0 + t, out = (uint64_t)n0 * 16 + col;
        if (token >= a.m || out >= a.n) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(&sh.y[0][t][col]);
#pragma unroll
        for (int w = 1; w < WK; ++w) v += *reinterpret_cast<const f32x4*>(&sh.y[w][t][col]);
        float f = O::FACTOR;
        if (a.xscale) f *= a.xscale[a.xscale_stride ? token : 0];
        store_y(a.y, a.y_type, token * a.y_stride + out, a.n - out, v * f);
    }
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, hipStream_t s) {
    // The widest workgroup of those that need the fewest turns of the compute
    // units: rounds of workgroups times the work of one.
    const uint64_t cus = (uint64_t)device_cu_count(), mblocks = tiles_of(a.m, MM_TOKENS);
    auto blocks = [&](int wn) { return mblocks * tiles_of(a.nt, 4 * wn); };
    auto turns = [&](int wn) { return (blocks(wn) + cus - 1) / cus * wn; };
    auto go = [&](auto wn) -> int {
        constexpr int WN = decltype(wn)::value;
        const uint64_t b = blocks(WN);
        if (b >= 1u << 31 || a.m >= 1u << 31) return LECB_ERR_TOO_LARGE;
        matmul_w4_kernel<X, S, GROUP, WN>
            <<<dim3((uint32_t)(b + 7) / 8 * 8), 64 * MM_WAVES, 0, s>>>(a, (uint32_t)mblocks, (uint32_t)b);
        return launched();
    };
    if (turns(8) <= turns(4)) return go(std::integral_constant<int, 8>());
    return go(std::integral_constant<int, 4>());
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

}  // namespace

int launch_matmul_w4(const MatvecArgs& a, int x_type, int scale_type, uint32_t group, hipStream_t s) {
    switch (x_type) {
        case LECB_I8: return launch_as<int8_t>(a, scale_type, group, s);
        case LECB_BF16: return launch_as<__bf16>(a, scale_type, group, s);
        default: return launch_as<_Float16>(a, scale_type, group, s);
    }
}

}  // namespace lecb
