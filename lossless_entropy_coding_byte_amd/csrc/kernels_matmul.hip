// Products of many tokens with 4-bit weights: y = x W^T (lecb.h gives the
// layout of W, kernels_matvec.hip the form for few tokens), and the layout of
// tokens that both take.
#include "matvec.hpp"

namespace lecb {

namespace {

// ---------------------------------------------------------------- tokens laid out

template <int CTRL>
__device__ inline float add_lanes(float v) {   // v + the v of the lane that CTRL names
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// A workgroup takes 16 tokens and the columns of 256 units: one tile of 16-bit
// tokens, two of bytes.  Lanes read along the tokens' rows and write along the
// pieces, through LDS (the XOR spreads both over the banks).
template <typename X>
__global__ __launch_bounds__(256) void lay_tokens_kernel(MatvecArgs a, uint32_t group, uint32_t across) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    constexpr int TILES = 16 / T::UNITS;
    __shared__ u32x4 sh[256];
    const uint32_t mt = blockIdx.x / across, tk0 = blockIdx.x % across * TILES, unit = threadIdx.x % T::UNITS, sub = threadIdx.x / T::UNITS % TILES;
    const uint32_t token = threadIdx.x / 16, tk = tk0 + sub;
    const uint64_t t = (uint64_t)mt * 16 + token, col = (uint64_t)tk * TILE_COLS;
    u32x4 v = {0, 0, 0, 0};
    if (t < a.m && tk < a.kt) {
        const X* p = reinterpret_cast<const X*>(a.x) + t * a.x_stride + col;
        v = O::order(col + TILE_COLS <= a.k ? T::load(p, unit) : T::load(p, unit, (uint32_t)(a.k - col)));
    }
    if constexpr (O::OFFSET) {
        // 16 neighbouring lanes hold a token's tile, group / 8 of them a group
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) s = O::dot(v[i], O::EXCESS, s);
        s = add_lanes<0xB1>(s);                     // the next lane's
        s = add_lanes<0x4E>(s);                     // the next two's
        if (group >= 64) s = add_lanes<0x141>(s);   // mirrored within eight
        if (group >= 128) s = add_lanes<0x140>(s);  // mirrored within sixteen
        const uint32_t per = group / 8, groups = 16 / per;
        if (tk < a.kt && unit % per == 0)
            laid_sums<X>(a)[((((uint64_t)(mt / 4) * a.kt + tk) * 4 + mt % 4) * groups + unit / per) * 16 + token] = s;
    }
    sh[(sub * T::UNITS + unit) * 16 + (token ^ unit)] = v;
    __syncthreads();
    const uint32_t u = threadIdx.x / 16, r = threadIdx.x % 16;   // unit of TILES tiles, token
    if (tk0 + u / T::UNITS < a.kt)
        reinterpret_cast<u32x4*>(a.ws)[((uint64_t)mt * a.kt + tk0) * (16 * T::UNITS) + threadIdx.x] =
            sh[u * 16 + (r ^ (u % T::UNITS))];
}

// ---------------------------------------------------------------- products

constexpr int MM_WAVES = 8;
constexpr int MM_ROWS = 64;   // of W, a wave's

// A workgroup takes 64 tokens and 64 WN rows of W; its eight waves are WN along
// the rows times 8 / WN along the columns.  A wave keeps 64 x 64 sums in
// registers: its words of W come from memory as the matrix instructions take
// them, become numbers there and serve four instructions each; the tokens come
// through LDS, where the WN waves of one share of the columns put each tile
// once, by loads that go there directly.
template <typename X, int GROUP>
struct MmTile {   // 64 tokens' tile
    u32x4 x[4 * Tokens<X>::PIECES][64];
    float excess[Operand<X>::OFFSET ? 64 * (128 / GROUP) : 4];   // [4][groups][16 tokens]
};

// Sends for one tile while the other is computed.  The compiler keeps the reads
// of `now` apart from the loads on their way to `next` for being told here that
// the two are different memory: it would wait for those loads first otherwise.
template <typename Tile, typename Fetch, typename Compute>
__device__ __forceinline__ void mm_step(const Tile* __restrict__ now, Tile* __restrict__ next, Fetch fetch, Compute compute) {
    fetch(next);
    compute(now);
}

template <typename X, typename S, int GROUP, int WN>
__global__ __launch_bounds__(64 * MM_WAVES) void matmul_w4_kernel(MatvecArgs a, uint32_t mblocks, uint32_t blocks) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    constexpr int WK = MM_WAVES / WN, GROUPS = 128 / GROUP, WORDS = GROUP / 32;
    constexpr int PIECES = 4 * T::PIECES;                  // of 64 tokens' tile
    constexpr int COLS = MM_ROWS * WN, PITCH = COLS + 4;   // outputs of a token; + 4: rows on other banks
    typedef MmTile<X, GROUP> Tile;
    union Shared {
        Tile tile[2][WK];
        float y[WK][LAID_TOKENS][PITCH];
    };
    __shared__ Shared sh;

    // Workgroups of one XCD (every eighth) take neighbouring rows of W, and the
    // blocks of tokens of the same rows are next to one another: what an XCD
    // reads of W it reads once.
    const uint32_t per = (blocks + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || id >= blocks) return;
    const uint32_t mb = id % mblocks, n0 = id / mblocks * (COLS / 16);   // 64 tokens, tile of W
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
    const u32x4* x = laid_tokens(a) + (uint64_t)mb * a.kt * (PIECES * 64);
    const float* excess = laid_sums<X>(a) + (uint64_t)mb * a.kt * (64 * GROUPS);

    u32x4 words[4], next_words[4];
    S scale[4][GROUPS], next_scale[4][GROUPS];
    auto fetch = [&](uint32_t tk, Tile* tile) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < PIECES / WN; ++q) {
            const uint32_t p = q * WN + wn;
            // piece p of the four blocks of 16 tokens, which lie a.kt tiles apart
            const u32x4* from = x + ((uint64_t)(p / T::PIECES) * a.kt + tk) * (T::PIECES * 64) + p % T::PIECES * 64;
            load_to_lds<16>(from + lane, tile->x[p]);
        }
        if constexpr (O::OFFSET) {
            if (wn == 0) {
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    load_to_lds<4>(excess + ((uint64_t)tk * GROUPS + g) * 64 + lane, tile->excess + 64 * g);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            next_words[j] = (tiles[j] + (uint64_t)tk * 64)[lane];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) next_scale[j][g] = (scales[j] + ((uint64_t)tk * GROUPS + g) * 16)[r];
        }
    };

    f32x4 sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = {0, 0, 0, 0};

    auto compute = [&](const Tile* tile) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            typename O::Acc acc[4][4];
            if constexpr (sizeof(X) == 1 && WORDS > 1) {
#pragma unroll
                for (int d = 0; d < WORDS; d += 2) {
                    u32x4 xo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) xo[i] = tile->x[i * T::PIECES + (g * WORDS + d) / 2][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x2 w0 = O::weights(words[j][g * WORDS + d]), w1 = O::weights(words[j][g * WORDS + d + 1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[i][j] = O::mul2(xo[i], w0, w1, d ? acc[i][j] : typename O::Acc{0, 0, 0, 0});
                    }
                }
            } else if constexpr (sizeof(X) == 1) {
                u32x2 xo[4];   // half a unit
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u32x4 v = tile->x[i * T::PIECES + g / 2][lane];
                    xo[i] = g & 1 ? u32x2{v.z, v.w} : u32x2{v.x, v.y};
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x2 w = O::weights(words[j][g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i][j] = O::mul(xo[i], w, typename O::Acc{0, 0, 0, 0});
                }
            } else {
                f32x4 over[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    over[i] = *reinterpret_cast<const f32x4*>(&tile->excess[(i * GROUPS + g) * 16 + 4 * c]);
#pragma unroll
                for (int d = 0; d < WORDS; ++d) {
                    u32x4 xo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) xo[i] = tile->x[i * T::PIECES + g * WORDS + d][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4 w = O::weights(words[j][g * WORDS + d]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i][j] = O::mul(xo[i], w, d ? acc[i][j] : over[i]);
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
            // four groups a tile: moving one's loads and words into another runs out of registers
            if (GROUPS == 4) __builtin_amdgcn_sched_barrier(0);
        }
    };

    // Every wave takes the same number of steps; those past the last tile only
    // wait.  A step's loads are in flight while the step before is computed.
    const uint32_t steps = (a.kt + WK - 1) / WK;
    if (wk < a.kt) fetch(wk, &sh.tile[0][wk]);
    for (uint32_t s = 0; s < steps; ++s) {
        const uint32_t tk = s * WK + wk;
        loads_done();
        lds_barrier();   // this tile is there, and the last one is read
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            words[j] = next_words[j];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) scale[j][g] = next_scale[j][g];
        }
        mm_step<Tile>(
            &sh.tile[s & 1][wk], &sh.tile[(s + 1) & 1][wk],
            [&](Tile* tile) __attribute__((always_inline)) { if (tk + WK < a.kt) fetch(tk + WK, tile); },
            [&](const Tile* tile) __attribute__((always_inline)) { if (tk < a.kt) compute(tile); });
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
    for (uint32_t at = threadIdx.x; at < LAID_TOKENS * COLS / 4; at += 64 * MM_WAVES) {
        const uint32_t t = at / (COLS / 4), col = at % (COLS / 4) * 4;
        const uint64_t token = (uint64_t)mb * LAID_TOKENS + t, out = (uint64_t)n0 * 16 + col;
        if (token >= a.m || out >= a.n) continue;
        f32x4 v = *reinterpret_cast<const f32x4*>(&sh.y[0][t][col]);
#pragma unroll
        for (int w = 1; w < WK; ++w) v += *reinterpret_cast<const f32x4*>(&sh.y[w][t][col]);
        store_y(a, token, out, v * O::FACTOR);
    }
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, hipStream_t s) {
    // The widest workgroup of those that need the fewest turns of the compute
    // units: rounds of workgroups times the work of one.
    const uint64_t cus = (uint64_t)device_cu_count(), mblocks = tiles_of(a.m, LAID_TOKENS);
    auto blocks = [&](int wn) { return mblocks * tiles_of(a.nt, 4 * wn); };
    auto turns = [&](int wn) { return (blocks(wn) + cus - 1) / cus * wn; };
    auto go = [&](auto wn) -> int {
        constexpr int WN = decltype(wn)::value;
        const uint64_t b = blocks(WN);
        if (b >= 1u << 31) return LECB_ERR_TOO_LARGE;
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

template <typename X>
int lay_as(const MatvecArgs& a, uint32_t group, uint64_t blocks, hipStream_t s) {
    const uint64_t across = tiles_of(a.kt, 16 / Tokens<X>::UNITS);
    if (blocks * across >= 1u << 31) return LECB_ERR_TOO_LARGE;
    lay_tokens_kernel<X><<<dim3((uint32_t)(blocks * across)), 256, 0, s>>>(a, group, (uint32_t)across);
    return launched();
}

}  // namespace

int launch_lay_tokens(const MatvecArgs& a, int x_type, uint32_t group, uint64_t blocks, hipStream_t s) {
    switch (x_type) {
        case LECB_I8: return lay_as<int8_t>(a, group, blocks, s);
        case LECB_BF16: return lay_as<__bf16>(a, group, blocks, s);
        default: return lay_as<_Float16>(a, group, blocks, s);
    }
}

int launch_matmul_w4(const MatvecArgs& a, int x_type, int scale_type, uint32_t group, hipStream_t s) {
    switch (x_type) {
        case LECB_I8: return launch_as<int8_t>(a, scale_type, group, s);
        case LECB_BF16: return launch_as<__bf16>(a, scale_type, group, s);
        default: return launch_as<_Float16>(a, scale_type, group, s);
    }
}

}  // namespace lecb
