// Attention over the 8-bit cache: the form for many rows (prompts).
#pragma once

#include "attend.hpp"

#if defined(__HIPCC__)
namespace lecb {

// Many rows: a workgroup takes 32 rows of one head a wave over a part of the
// tiles, two at a time.  Their codes are turned into halves once, by all waves,
// and put into LDS as matrix operands of 1 KiB: of keys for 32 tokens x 16
// dimensions, of values for 32 dimensions x 16 tokens, each in the order of the
// lanes.  Matrix instructions by 32 x 32 x 16, transposed as in the form for few
// rows: a row's scores stand in two lanes, which is the second product's operand,
// with tokens 16 m + 8 (i / 4) + 4 (lane / 32) + i % 4 as its eight, so the
// values' operands are put together in that order.
//
// Bound by instruction issue: of a tile and 32 rows, 512 cycles of products stand
// beside some 600 of vector instructions, a third of them exponentials and a
// fifth (a tenth with eight waves) codes to halves.  512 tokens after 32256, 32 heads to 8 of 128
// dimensions: 300 us, 910 TFLOP/s, the matrix units busy 42 % of the time (four waves
// and two workgroups a compute unit 323), 460 in fp16 and 710 in fp32 with their weights' and queries' parts;
// two prompts of up to 4096 tokens 276 with the other launches, 660.  Dimensions of 96
// have three units, which eight waves do not share evenly; more than 128, or 32 bits, need
// the registers of two waves.  Tried and slower: 64 rows a wave (half the reads of LDS, but one
// wave a SIMD, and sums outside of the vector registers: 340 -> 399 us), all products of a step
// in one go after its softmax (332 -> 364).
template <typename T, int U>
constexpr int MANY_WAVES = U <= 4 && U != 3 && sizeof(T) == 2 ? 8 : 4;
template <typename T, int U>
constexpr int MANY_ROWS = 32 * MANY_WAVES<T, U>;

template <typename T, int U>
struct ManyMemory {
    union {
        struct {
            uint8_t k[2][2][2 * U][UNIT_BYTES];    // [buffer][tile][16 dimensions]
            uint8_t v[3][2][U][2][UNIT_BYTES];     // [buffer][tile][32 dimensions][16 tokens]
        };
        T rows[MANY_ROWS<T, U>][32 * U];   // queries before, results after
    };
};

template <typename T, int U>
__device__ inline void attend_many(const AttendArgs& a, const Item& it, uint32_t h, ManyMemory<T, U>& mem) {
    constexpr int WAVES = MANY_WAVES<T, U>, ROWS = MANY_ROWS<T, U>, SHARE = 4 * U / WAVES, NQ = Parts<T>::Q, NP = Parts<T>::P;
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, hh = lane >> 5;
    Work k;
    if (!work_of<ROWS>(a, it, h, k)) return;
    if (k.bad) {
        bad_rows<T>(a, k, h);
        return;
    }
    const uint32_t seq = it.seq;

    // rows: lane r of each 32 has row r of the wave's, dimensions 16 e + 8 hh and on
    stage_rows(a, k, h, ROWS, 32 * U, &mem.rows[0][0]);
    __syncthreads();
    const uint32_t mine = 32 * wave + r, row = k.r0 + mine;
    f16x8 q[2 * U][NQ];
    const Factor factor = load_row<T, 2 * U, 32>(a, mem.rows[mine], 8 * hh, 16, q);
    const int pos = k.old + (row < k.rows ? (int)(row / a.group) : 0);
    const int hi = a.causal ? pos : k.len - 1, lo = a.window ? pos - (int)a.window + 1 : 0;
    __syncthreads();
    // tiles go by pairs: what a pair has too many is masked
    const int from = k.from, to = k.to, lo_most = k.lo_most, hi_least = k.hi_least;
    const uint32_t shift = __builtin_ctz(a.seqs.block / TILE_TOKENS);

    f32x16 acc[U];
    float ref = inf(), sum = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[u][i] = 0.0f;

    // the blocks of a step's tiles t and t + 1, in even and odd lanes
    auto pages = [&](int t) { return a.seqs.page(seq, ((uint32_t)t + (lane & 1)) >> shift); };
    // their scales: keys' in lanes 0 and 1, values' in 2 and 3
    auto load_scales = [&](uint32_t found) {
        return (lane & 2 ? a.v_scale : a.k_scale)[(uint64_t)(found < a.seqs.blocks ? found : 0) * a.heads + h];
    };
    // a wave's share of a step's codes: keys or values of one tile, all units of it or half of them
    const bool keys = !(wave & 2);
    const uint32_t u0 = wave / 4 * SHARE;
    auto load_codes = [&](uint32_t found, int t, u32x4 (&w)[SHARE]) {
        const uint32_t page = of_lane(found, wave & 1);
        const uint64_t cell = (uint64_t)(page < a.seqs.blocks ? page : 0) * a.heads + h;
        const uint64_t at = ((cell << shift) + (((uint32_t)t + (wave & 1)) & ((1u << shift) - 1))) * (U * UNIT_BYTES) + u0 * UNIT_BYTES + lane * 16;
        const uint8_t* codes = keys ? a.k : a.v;
#pragma unroll
        for (int u = 0; u < SHARE; ++u) w[u] = *reinterpret_cast<const u32x4*>(codes + at + u * UNIT_BYTES);
    };
    // and into LDS, as operands
    auto put = [&](const u32x4 (&w)[SHARE], int kb, int vb) {
        const uint32_t tile = wave & 1, g = lane >> 4;
        if (keys) {
            // lane 16 g + t: dimensions 32 u + 8 g of tokens t and 16 + t
            const uint32_t at = ((g & 1) * 32 + (lane & 15)) * 16;
#pragma unroll
            for (int u = 0; u < SHARE; ++u) {
                uint8_t* p = mem.k[kb][tile][2 * (u0 + u) + (g >> 1)] + at;
                *reinterpret_cast<f16x8*>(p) = operand(w[u][0], w[u][1]);
                *reinterpret_cast<f16x8*>(p + 16 * 16) = operand(w[u][2], w[u][3]);
            }
        } else {
            // lane 16 g + d: tokens 4 g, then 16 + 4 g, of dimensions d, then 16 + d
            const uint32_t at = ((g & 1) * 32 + (lane & 15)) * 16 + (g >> 1) * 8;
#pragma unroll
            for (int u = 0; u < SHARE; ++u)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t v[2];
                        halves(w[u][2 * b + m], v);
                        *reinterpret_cast<u32x2*>(mem.v[vb][tile][u0 + u][m] + at + b * 16 * 16) = u32x2{v[0], v[1]};
                    }
        }
    };
    auto scores = [&](f32x16& s, int kb, int tile) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
            const f16x8 codes = *reinterpret_cast<const f16x8*>(mem.k[kb][tile][u] + lane * 16);
#pragma unroll
            for (int j = 0; j < NQ; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes, q[u][j], s, 0, 0, 0);
        }
    };
    // masks, and the running maximum; what takes scores and weights further.  A weight of one part
    // comes out of the exponential times the values' scale, to 2^-23 of the scale's logarithm, and its
    // sum takes the scale off again.  That holds where the scale is a number that the reciprocal
    // reaches and no more than 2^60 below the largest so far (the exponential's range then leaves 77 bits
    // below equal weights of that block); other scales, of either sign and zero, are multiplied in after the sum.
    float f, lift = 0.0f, up = 1.0f;
    bool odd = false;
    uint32_t high = 0;   // the bits of the largest scale so far
    auto begin = [&](f32x16& s, int t, float ks, float vs) {
        const int at = t * (int)TILE_TOKENS;
        f = factor.times(ks);
        // all rows see all of the tile's tokens, and the larger product is the larger score; or not
        if (!(at >= lo_most && at + (int)TILE_TOKENS - 1 <= hi_least && a.scale >= 0.0f && ks >= 0.0f)) {
            asm volatile("");   // not to be done and then selected from
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int token = at + 8 * (e / 4) + 4 * (int)hh + e % 4;
                s[e] = token <= hi && token >= lo ? s[e] * f : -inf();
            }
            f = 1.0f;
        }
        const bool number = fabsf(vs) < inf();
        if constexpr (NP == 1) {
            // in scalar registers: 2^-60 to 2^100, and 2^60 over the bits' exponent
            const uint32_t bits = __float_as_uint(vs), size = bits & 0x7fffffffu;
            if (size < 0x7f800000u && size > high) high = size;
            odd = bits - 0x21800000u > 0x71800000u - 0x21800000u || size + (60u << 23) < high;
            lift = odd ? 0.0f : __builtin_amdgcn_logf(vs) + P_DOWN_LOG2;
            up = odd ? 1.0f : OUT * __builtin_amdgcn_rcpf(vs);
        }
        float m = -inf();
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, s[e]);
        m = max_of_halves(m * f);
        // values without a number to scale them: no number to the rows that see one of them
        if (!number && m != -inf()) sum = __uint_as_float(0x7fc00000u);
        const float next = REF_TOP - (m + scale_exponent(vs));
        if (__ballot(next < ref - LAG)) {
            const float root = next < ref ? root_of(next - ref) : 1.0f, down_by = root * root;
            sum = sum * root * root;
#pragma unroll
            for (int u = 0; u < U; ++u) acc[u] *= down_by;
            ref = fminf(ref, next);
        }
    };
    auto finish = [&](f32x16& s, int vb, int tile, float vs) {
        const float base = (ref == inf() ? 0.0f : ref) + lift;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            f16x8 p[NP];
            float part = 0.0f;
#pragma unroll
            for (int e = 8 * m; e < 8 * m + 8; ++e) {
                s[e] = exp2_of(fmaf(s[e], f, base));
                part += s[e];
                if (NP > 1) s[e] = product(s[e], fabsf(vs) < inf() ? vs * P_DOWN : 0.0f);
            }
            sum = NP == 1 ? fmaf(part, up, sum) : sum + part;
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[j][e] = (_Float16)s[8 * m + e];
                    if (NP > 1) s[8 * m + e] -= (float)p[j][e];
                }
            if (NP == 1 && odd) {
                asm volatile("");   // not to be done and then selected from
                const float down = fabsf(vs) < inf() ? vs * P_DOWN : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) p[0][e] = (_Float16)(s[8 * m + e] * down);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const f16x8 codes = *reinterpret_cast<const f16x8*>(mem.v[vb][tile][u][m] + lane * 16);
#pragma unroll
                for (int j = 0; j < NP; ++j) acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes, p[j], acc[u], 0, 0, 0);
            }
        }
    };

    if (from < to) {
        // Of each tile, its scores' products are issued among the exponentials of the one before,
        // whose own products with the values follow.  A step is two tiles: the next step's codes go
        // into LDS in its first half, those after them are asked for, blocks are looked up one
        // more ahead.  Past the last step the same again.
        auto next_of = [&](int t) { return t + 2 < to ? t + 2 : t; };
        int t1 = next_of(from), t2 = next_of(t1);
        uint32_t found = pages(from), found1 = pages(t1);
        u32x4 w[SHARE];
        load_codes(found, from, w);
        float scales = load_scales(found);
        put(w, 0, 0);
        load_codes(found1, t1, w);
        float scales1 = load_scales(found1);
        uint32_t found2 = pages(t2);
        __syncthreads();
        f32x16 s0, s1;
        scores(s0, 0, 0);
        int kb = 0, vb = 0;
        for (int t = from; t < to; t += 2) {
            const float keys_scales = key_scale(scales, found < a.seqs.blocks);
            const float ks0 = of_lane(keys_scales, 0), vs0 = of_lane(scales, 2);
            const float ks1 = of_lane(keys_scales, 1), vs1 = of_lane(scales, 3);
            const int vn = vb == 2 ? 0 : vb + 1;
            begin(s0, t, ks0, vs0);
            scores(s1, kb, 1);
            finish(s0, vb, 0, vs0);
            put(w, kb ^ 1, vn);
            load_codes(found2, t2, w);
            found = found1;
            scales = scales1;
            scales1 = load_scales(found2);
            found1 = found2;
            t2 = next_of(t2);
            found2 = pages(t2);
            __syncthreads();
            begin(s1, t + 1, ks1, vs1);
            kb ^= 1;
            scores(s0, kb, 0);
            finish(s1, vb, 1, vs1);
            vb = vn;
        }
        __syncthreads();
    }

    sum += __shfl_xor(sum, 32);
    if (k.parts > 1) {
        if (mine >= k.have) return;
        float* ws = form_of<ROWS>(a).ws + ((uint64_t)k.slot * ROWS + mine) * (32 * U + 4);
        if (hh == 0) {
            ws[0] = ref;
            ws[1] = sum;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4*>(ws + 4 + 32 * u + 8 * j + 4 * hh) =
                    f32x4{acc[u][4 * j], acc[u][4 * j + 1], acc[u][4 * j + 2], acc[u][4 * j + 3]};
        return;
    }
    // through LDS, so that rows leave whole
    typedef T four __attribute__((ext_vector_type(4)));
    const float over = sum == 0.0f ? 0.0f : OUT / sum;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<four*>(&mem.rows[mine][32 * u + 8 * j + 4 * hh]) =
                four{(T)(acc[u][4 * j] * over), (T)(acc[u][4 * j + 1] * over), (T)(acc[u][4 * j + 2] * over),
                     (T)(acc[u][4 * j + 3] * over)};
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < k.have * (8 * U); i += blockDim.x) {
        const uint32_t row = i / (8 * U), d = i % (8 * U) * 4;
        if (d >= a.dim) continue;
        const four x = *reinterpret_cast<const four*>(&mem.rows[row][d]);
        const T o[4] = {x[0], x[1], x[2], x[3]};
        put_four(a, k, h, k.r0 + row, d, o);
    }
}

}  // namespace lecb
#endif
