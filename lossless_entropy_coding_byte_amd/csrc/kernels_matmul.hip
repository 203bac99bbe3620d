// Products of many tokens with 4-bit weights: y = x W^T (lecb.h gives the
// layout of W, kernels_matvec.hip the form for few tokens), and the layout of
// tokens that both take.
#include "matvec.hpp"

namespace lecb {

namespace {

// ---------------------------------------------------------------- tokens laid out

// A workgroup takes 16 tokens and the columns of 256 units: one tile of 16-bit
// tokens, two of bytes.  Lanes read along the tokens' rows and write along the
// pieces, through LDS (the XOR spreads both over the banks).
//
// What the products gain from it: whole, aligned loads of 1 KiB where rows of a
// power of two bytes apart would come from one memory channel, sixteen at a time
// (32 x 8192 x 8192 int8: 19 us without, 12.8 with), no partial tiles, and the
// order of the tokens made once instead of by every workgroup.  Bound by latency:
// 512 x 8192 bf16 6 us, 32 x 8192 int8 2.7 us.
template <typename X, bool MANY>
__global__ __launch_bounds__(256) void lay_tokens_kernel(MatvecArgs a, uint32_t first, uint32_t across) {
    typedef Operand<X> O;
    typedef Tokens<X> T;
    constexpr int TILES = 16 / T::UNITS;
    __shared__ u32x4 sh[256];
    const uint32_t mt = blockIdx.x / across, tk0 = (first + blockIdx.x % across) * TILES;
    const uint32_t unit = threadIdx.x % T::UNITS, sub = threadIdx.x / T::UNITS % TILES;
    const uint32_t token = threadIdx.x / 16, tk = tk0 + sub;
    const uint64_t t = (uint64_t)mt * 16 + token, col = (uint64_t)tk * TILE_COLS;
    u32x4 v = {0, 0, 0, 0};
    if (t < a.m && tk < a.kt) {
        const X* p = reinterpret_cast<const X*>(a.x) + t * a.x_stride + col;
        v = O::order(col + TILE_COLS <= a.k ? T::load(p, unit) : T::load(p, unit, (uint32_t)(a.k - col)));
    }
    sh[(sub * T::UNITS + unit) * 16 + (token ^ unit)] = v;
    __syncthreads();
    const uint32_t u = threadIdx.x / 16, r = threadIdx.x % 16;   // unit of TILES tiles, token
    const uint32_t tk1 = tk0 + u / T::UNITS, u1 = u % T::UNITS;
    if (tk1 >= a.kt) return;
    // MANY: piece 2 p + s, lane 32 h + (mt odd: 16) + r, for unit 4 p + 2 h + s
    const uint64_t at = MANY ? ((uint64_t)(mt / 2) * a.kt + tk1) * (32 * T::UNITS) + (u1 / 4 * 2 + u1 % 2) * 64 +
                                   u1 / 2 % 2 * 32 + mt % 2 * 16 + r
                             : ((uint64_t)mt * a.kt + tk1) * (16 * T::UNITS) + u1 * 16 + r;
    reinterpret_cast<u32x4*>(a.ws)[at] = sh[u * 16 + (r ^ u1)];
}

// ---------------------------------------------------------------- products

constexpr int MM_WAVES = 8;
constexpr int MM_ROWS = 64;   // of W, a wave's

// What a share of the columns has in LDS of one tile of 128 columns: 64 tokens
// and 64 WN rows of W.
template <typename X, typename S, int GROUP, int WN>
struct MmTile {
    static constexpr int GROUPS = 128 / GROUP, PIECES = 2 * Tokens<X>::PIECES;
    static constexpr int SCALES = GROUPS * 4 * 16, LOADS = SCALES * sizeof(S) < 256 ? 1 : SCALES * sizeof(S) / 256;
    u32x4 x[2 * PIECES][64];
    S scales[WN][LOADS * 256 / sizeof(S)];                // [4][groups][16 rows]
};

// Sends for a tile while another is computed.  The compiler keeps the reads
// of `now` apart from the loads on their way to `next` for being told here that
// the two are different memory: it would wait for those loads first otherwise.
template <typename Tile, typename F>
__device__ __forceinline__ void mm_step(const Tile* __restrict__ now, Tile* __restrict__ next, F f) {
    f(now, next);
}

// A workgroup takes 64 tokens and 64 WN rows of W; its eight waves are WN along
// the rows times 8 / WN along the columns.  A wave keeps 64 x 64 sums in
// registers.  Everything comes through LDS, by loads that go there directly and
// are sent one tile ahead: a share's tokens once for its WN waves, each wave's
// own words and scales.  Products go by 32 tokens x 32 rows: beside matrix
// instructions a SIMD sends one vector instruction in about 4.5 cycles, so their
// number is what counts, and these take half as many as 16 x 16 ones.
//
// Bound by that issue: of 16-bit tokens, a tile of 128 columns costs a wave 32
// matrix instructions (1024 cycles), about 280 vector ones (208 for its words,
// 64 a group for the scales) and 90 others.  512 x 8192 x 8192 bf16: groups of 128
// 70 us, 980 TFLOP/s, of 64 75, of 32 86; int8, groups of 128, 46 us.  With the layout
// of the tokens, on a slower card: 80, 81 and 94; operands with an offset (Operand),
// which eight instructions a word make instead of 13 but whose sums are read from
// LDS for every group, 77, 88 and 99 there (the library's product of two bf16
// matrices of 8192 x 8192: 1250 TFLOP/s).  Tried and slower: one matrix
// instruction, then a share of the vector ones, in turn (+ 15 %, as then neither
// wave of a SIMD runs ahead); all words' numbers before all products (registers);
// a wave's words through LDS (its reads are the bound).
template <typename X, typename S, int GROUP, int WN>
__global__ __launch_bounds__(64 * MM_WAVES) void matmul_w4_kernel(MatvecArgs a, uint32_t mblocks, uint32_t blocks) {
    typedef Operand<X> O;
    typedef MmTile<X, S, GROUP, WN> Tile;
    constexpr int WK = MM_WAVES / WN, GROUPS = 128 / GROUP, WORDS = GROUP / 32, PIECES = Tile::PIECES;
    constexpr int COLS = MM_ROWS * WN, PITCH = COLS + 8;   // outputs of a token; + 8: rows on other banks
    union Shared {
        Tile tile[3][WK];
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
    const uint32_t lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;

    // tiles past the last repeat it: their sums are not stored
    auto tile_row = [&](uint32_t j) -> uint64_t { return n0 + wn * 4 + j < a.nt ? n0 + wn * 4 + j : a.nt - 1; };
    // lane 32 h + r's words: row r of 32, columns 32 d + 16 h + 8 s ..
    const u32x4* from_words[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) from_words[j] = a.tiles + tile_row(2 * j + r / 16) * a.kt * 64 + 32 * h + r % 16;
    struct Words {
        u32x4 v[2][2];
    } words0, words1;
    // the wave's four tiles' scales, four bytes a lane; within 4 GiB of the first's (kt < MM_TILES)
    constexpr uint32_t ROW = GROUPS * 16 * sizeof(S);
    static_assert(3ull * MM_TILES * ROW < 1ull << 32, "offsets of scales");
    const char* from_scales = reinterpret_cast<const char*>(a.scales) + tile_row(0) * a.kt * ROW;
    uint32_t scale_offset[Tile::LOADS];
#pragma unroll
    for (int q = 0; q < Tile::LOADS; ++q) {
        const uint32_t b = (q * 256 + lane * 4) % (4 * ROW);
        scale_offset[q] = (uint32_t)(tile_row(b / ROW) - tile_row(0)) * a.kt * ROW + b % ROW;
    }
    const u32x4* from_x = laid_tokens(a) + (uint64_t)mb * a.kt * (2 * PIECES * 64);

    auto fetch_words = [&](Words& w, uint32_t tk) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int s = 0; s < 2; ++s) w.v[j][s] = from_words[j][(uint64_t)tk * 64 + s * 16];
        asm volatile("" ::: "memory");   // here, not where they are needed
    };
    constexpr int SENDS = 2 * PIECES / WN + Tile::LOADS;
    auto send = [&](uint32_t tk, Tile* tile, int i) __attribute__((always_inline)) {
        constexpr int A = 2 * PIECES / WN;
        if (i < A) {
            // piece p of the two blocks of 32 tokens, which lie a.kt tiles apart
            const uint32_t p = i * WN + wn;
            load_to_lds<16>(from_x + ((uint64_t)(p / PIECES) * a.kt + tk) * (PIECES * 64) + p % PIECES * 64, 16 * lane,
                            tile->x[p]);
        } else {
            load_to_lds<4>(from_scales + (uint64_t)tk * ROW, scale_offset[i - A],
                           &tile->scales[wn][(i - A) * (256 / sizeof(S))]);
        }
    };

    f32x16 sum[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[i][j][e] = 0.0f;

    // A group's columns, then 32 rows of W: those words become numbers and the
    // rows before are scaled while the matrix instructions run.
    auto step = [&](uint32_t tk, const Words& words, Words& next_words, const Tile* now, Tile* next) __attribute__((always_inline)) {
        const uint32_t ahead = tk + 2 * WK < a.kt ? tk + 2 * WK : a.kt - 1;   // past the last: sent again, not used
        typedef decltype(O::mul32({}, {}, {})) Acc;
        constexpr int N = sizeof(X) == 2 ? 2 * WORDS : WORDS == 1 ? 2 : WORDS;   // pieces of a group
        constexpr int UNITS = 2 * GROUPS;
        fetch_words(next_words, tk + WK < a.kt ? tk + WK : a.kt - 1);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            u32x4 xo[2][N];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < N; ++p)
                    xo[i][p] = now->x[i * PIECES + (sizeof(X) == 1 && WORDS == 1 ? g / 2 * 2 : g * N) + p][lane];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int q = 0; q < SENDS; ++q)   // spread over the units
                    if (q * UNITS / SENDS == g * 2 + j) send(ahead, next, q);
                Acc acc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][e] = 0;
                if constexpr (sizeof(X) == 2) {
#pragma unroll
                    for (int p = 0; p < N; ++p) {
                        const u32x4 w = O::weights(words.v[j][p % 2][g * WORDS + p / 2]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) acc[i] = O::mul32(xo[i][p], w, acc[i]);
                    }
                } else if constexpr (WORDS == 1) {   // half a unit
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const u32x2 w = O::weights(words.v[j][p][g]);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            acc[i] = O::mul32(g & 1 ? u32x2{xo[i][p].z, xo[i][p].w} : u32x2{xo[i][p].x, xo[i][p].y}, w, acc[i]);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < N; ++p) {
                        const u32x2 w0 = O::weights(words.v[j][p % 2][g * WORDS + p / 2 * 2]);
                        const u32x2 w1 = O::weights(words.v[j][p % 2][g * WORDS + p / 2 * 2 + 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) acc[i] = O::mul32x2(xo[i][p], w0, w1, acc[i]);
                    }
                }
                const float s = (float)now->scales[wn][((2 * j + r / 16) * GROUPS + g) * 16 + r % 16] * O::SCALE;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[i][j][e] = fmaf((float)acc[i][e], s, sum[i][j][e]);
            }
        }
    };

    // Every wave takes the same number of steps; those past the last tile only
    // wait.  Tokens are sent for two tiles ahead, words fetched for one: when
    // the words are there, all that was sent before them is too.
    const uint32_t steps = (a.kt + WK - 1) / WK;
    if (wk < a.kt) {
#pragma unroll
        for (int q = 0; q < SENDS; ++q) send(wk, &sh.tile[0][wk], q);
        fetch_words(words0, wk);
#pragma unroll
        for (int q = 0; q < SENDS; ++q) send(wk + WK < a.kt ? wk + WK : a.kt - 1, &sh.tile[1][wk], q);
    }
    uint32_t tk = wk, b = 0;
    auto turn = [&](const Words& words, Words& next_words) __attribute__((always_inline)) {
        loads_done<SENDS>();
        lds_barrier();   // this tile is there, and the last one is read
        if (tk < a.kt)
            mm_step<Tile>(&sh.tile[b][wk], &sh.tile[b == 0 ? 2 : b - 1][wk],
                          [&](const Tile* now, Tile* next) __attribute__((always_inline)) { step(tk, words, next_words, now, next); });
        tk += WK;
        b = b == 2 ? 0 : b + 1;
    };
    for (uint32_t s = 0; s < steps; s += 2) {
        turn(words0, words1);
        if (s + 1 < steps) turn(words1, words0);
    }

    // The columns' shares are added up in a fixed order, and a lane stores four
    // neighbouring outputs.
    loads_done<0>();
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sh.y[wk][32 * i + e / 4 * 8 + 4 * h + e % 4][wn * MM_ROWS + 32 * j + r] = sum[i][j][e];
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

// Rounds of workgroups on the compute units times the work of one.
uint64_t turns(const MatvecArgs& a, int wn) {
    const uint64_t cus = (uint64_t)device_cu_count();
    return (tiles_of(a.m, LAID_TOKENS) * tiles_of(a.nt, 4 * wn) + cus - 1) / cus * wn;
}

template <typename X, typename S, int GROUP>
int launch_group(const MatvecArgs& a, hipStream_t s) {
    // The wider workgroup unless it needs more turns.
    const uint64_t mblocks = tiles_of(a.m, LAID_TOKENS);
    auto go = [&](auto wn) -> int {
        constexpr int WN = decltype(wn)::value;
        const uint64_t b = mblocks * tiles_of(a.nt, 4 * WN);
        matmul_w4_kernel<X, S, GROUP, WN>
            <<<dim3((uint32_t)(b + 7) / 8 * 8), 64 * MM_WAVES, 0, s>>>(a, (uint32_t)mblocks, (uint32_t)b);
        return launched();
    };
    if (turns(a, 8) <= turns(a, 4)) return go(std::integral_constant<int, 8>());
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
int lay_as(const MatvecArgs& a, bool many, hipStream_t s) {
    const uint64_t across = tiles_of(a.kt, 16 / Tokens<X>::UNITS);
    const uint64_t down = many ? tiles_of(a.m, LAID_TOKENS) * (LAID_TOKENS / 16) : tiles_of(a.m, 16);
    for (uint64_t first = 0; first < across; first += LAY_ACROSS) {
        const uint32_t here = (uint32_t)(across - first < LAY_ACROSS ? across - first : LAY_ACROSS);
        const dim3 grid((uint32_t)(here * down));
        if (many)
            lay_tokens_kernel<X, true><<<grid, 256, 0, s>>>(a, (uint32_t)first, here);
        else
            lay_tokens_kernel<X, false><<<grid, 256, 0, s>>>(a, (uint32_t)first, here);
        const int rc = launched();
        if (rc) return rc;
    }
    return LECB_OK;
}

}  // namespace

uint64_t matmul_w4_turns(const MatvecArgs& a) {
    const uint64_t a8 = turns(a, 8), a4 = turns(a, 4);
    return a8 < a4 ? a8 : a4;
}

int launch_lay_tokens(const MatvecArgs& a, int x_type, bool many, hipStream_t s) {
    switch (x_type) {
        case LECB_I8: return lay_as<int8_t>(a, many, s);
        case LECB_BF16: return lay_as<__bf16>(a, many, s);
        default: return lay_as<_Float16>(a, many, s);
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
