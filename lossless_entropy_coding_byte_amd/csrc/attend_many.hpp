// Attention over the 8-bit cache: the form for many rows (prompts).
#pragma once

#include "attend.hpp"

#if defined(__HIPCC__)
namespace lecb {

// A wave's part of a step of two tiles: wave w loads the units of one tile's keys
// (w < 2) or values.
template <int U>
struct Part {
    u32x4 w[U];
    float scales;      // of the tiles' keys in lanes 0 and 1, of their values in 2 and 3
    uint32_t pages;    // of the tiles, in even and odd lanes: 0xffffffff where there is none
    __device__ void load(const AttendArgs& a, uint32_t found, uint32_t t, uint32_t shift, uint32_t h, uint32_t wave,
                         uint32_t lane) {
        pages = found;
        const uint32_t page = of_lane(found, wave & 1), mine = found < a.seqs.blocks ? found : 0;
        const uint64_t cell = (uint64_t)(page < a.seqs.blocks ? page : 0) * a.heads + h;
        const uint64_t at = ((cell << shift) + ((t + (wave & 1)) & ((1u << shift) - 1))) * (U * UNIT_BYTES) + lane * 16;
        const uint8_t* codes = wave < 2 ? a.k : a.v;
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = *reinterpret_cast<const u32x4*>(codes + at + u * UNIT_BYTES);
        scales = (lane & 2 ? a.v_scale : a.k_scale)[(uint64_t)mine * a.heads + h];
    }
};
struct Scales {
    float k[2], v[2];
    template <int U>
    __device__ void set(const AttendArgs& a, const Part<U>& x) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            k[i] = of_lane(x.pages, i) < a.seqs.blocks ? of_lane(x.scales, i) : __uint_as_float(0x7fc00000u);
            v[i] = of_lane(x.scales, 2 + i);
        }
    }
};

// Many rows: a workgroup takes 128 rows of one head, 32 a wave, over a part of the
// tiles, two at a time.  Their codes are turned into halves once, by all waves, and
// put into LDS as matrix operands of 1 KiB: of keys for 32 tokens x 16
// dimensions, of values for 32 dimensions x 16 tokens, each in the order of the
// lanes.  Matrix instructions by 32 x 32 x 16, transposed as in the form for few
// rows: a row's scores stand in two lanes, which is the second product's operand,
// with tokens 16 m + 8 (i / 4) + 4 (lane / 32) + i % 4 as its eight, so the
// values' operands are put together in that order.
template <typename T, int U>
struct ManyMemory {
    union {
        struct {
            uint8_t k[2][2][2 * U][UNIT_BYTES];    // [buffer][tile][16 dimensions]
            uint8_t v[2][2][U][2][UNIT_BYTES];     // [buffer][tile][32 dimensions][16 tokens]
        };
        T rows[MANY_ROWS][32 * U];   // queries before, results after
    };
};

template <typename T, int U>
__device__ inline void attend_many(const AttendArgs& a, const Item& it, uint32_t h, ManyMemory<T, U>& mem) {
    constexpr int ROWS = MANY_ROWS, NQ = Parts<T>::Q, NP = Parts<T>::P;
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, hh = lane >> 5;
    Work k;
    if (!work_of<ROWS>(a, it, h, k)) return;
    if (k.bad) {
        bad_rows<T>(a, k, h);
        return;
    }
    const uint32_t seq = it.seq;

    // rows: lane r of each 32 has row r of the wave's, dimensions 16 e + 8 hh and on
    const uint32_t row = k.r0 + 32 * wave + r;
    const bool real = row < k.rows;
    f16x8 q[2 * U][NQ];
    stage_rows(a, k, h, ROWS, 32 * U, &mem.rows[0][0]);
    __syncthreads();
    const float factor = load_row<T, 2 * U, 32>(a, mem.rows[32 * wave + r], 8 * hh, 16, q);
    __syncthreads();
    const int at_token = k.old + (real ? (int)(row / a.group) : 0);
    const int hi = a.causal ? at_token : k.len - 1, lo = a.window ? at_token - (int)a.window + 1 : 0;
    // tiles go by pairs: what a pair has too many is masked
    const int from = k.from, to = k.to, lo_most = k.lo_most, hi_least = k.hi_least;
    const uint32_t shift = __builtin_ctz(a.seqs.block / TILE_TOKENS);

    f32x16 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[u][i] = 0.0f;
    float ref = inf(), sum = 0.0f;

    // the blocks of tiles t and t + 1, in even and odd lanes
    auto pages = [&](int t) { return a.seqs.page(seq, ((uint32_t)t + (lane & 1)) >> shift); };
    // a wave's units into LDS, as operands
    auto put = [&](const Part<U>& x, int buf) {
        const uint32_t tile = wave & 1;
        if (wave < 2) {
            // lane 16 g + t: dimensions 32 u + 8 g of tokens t and 16 + t
            const uint32_t g = lane >> 4, at = ((g & 1) * 32 + (lane & 15)) * 16;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint8_t* p = mem.k[buf][tile][2 * u + (g >> 1)] + at;
                *reinterpret_cast<f16x8*>(p) = operand(x.w[u][0], x.w[u][1]);
                *reinterpret_cast<f16x8*>(p + 16 * 16) = operand(x.w[u][2], x.w[u][3]);
            }
        } else {
            // lane 16 g + d: tokens 4 g, then 16 + 4 g, of dimensions d, then 16 + d
            const uint32_t g = lane >> 4, at = ((g & 1) * 32 + (lane & 15)) * 16 + (g >> 1) * 8;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t v[2];
                        halves(x.w[u][2 * b + m], v);
                        *reinterpret_cast<u32x2*>(mem.v[buf][tile][u][m] + at + b * 16 * 16) = u32x2{v[0], v[1]};
                    }
        }
    };
    auto compute = [&](int t, int buf, const Scales& c) {
        f32x16 s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[i][e] = 0.0f;
#pragma unroll
            for (int u = 0; u < 2 * U; ++u) {
                const f16x8 codes = *reinterpret_cast<const f16x8*>(mem.k[buf][i][u] + lane * 16);
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes, q[u][j], s[i], 0, 0, 0);
            }
        }
        const int at = t * (int)TILE_TOKENS;
        float f[2] = {factor * c.k[0], factor * c.k[1]}, most = -inf();
        // all rows see all of the tiles' tokens, and the larger product is the larger score; or not
        if (!(at >= lo_most && at + 2 * (int)TILE_TOKENS - 1 <= hi_least && a.scale >= 0.0f && c.k[0] >= 0.0f && c.k[1] >= 0.0f)) {
            asm volatile("");   // not to be done and then selected from
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int pos = at + i * (int)TILE_TOKENS + 8 * (e / 4) + 4 * (int)hh + e % 4;
                    s[i][e] = pos <= hi && pos >= lo ? s[i][e] * f[i] : -inf();
                }
                f[i] = 1.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float m = -inf();
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, s[i][e]);
            m = max_of_halves(m * f[i]);
            most = fmaxf(most, m + scale_exponent(c.v[i]));
            // values without a number to scale them: no number to the rows that see one of them
            if (!(fabsf(c.v[i]) < inf()) && m != -inf()) sum = __uint_as_float(0x7fc00000u);
        }
        const float next = REF_TOP - most;
        if (__ballot(next < ref - LAG)) {
            const float down_by = next < ref ? exp2_of(next - ref) : 1.0f;
            sum *= down_by;
#pragma unroll
            for (int u = 0; u < U; ++u) acc[u] *= down_by;
            ref = fminf(ref, next);
        }
        const float base = ref == inf() ? 0.0f : ref;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float down = fabsf(c.v[i]) < inf() ? c.v[i] * P_DOWN : 0.0f;
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[i][e] = exp2_of(fmaf(s[i][e], f[i], base));
                part += s[i][e];
                s[i][e] *= down;
            }
            sum += part;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                f16x8 p[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[j][e] = (_Float16)s[i][8 * m + e];
                        s[i][8 * m + e] -= (float)p[j][e];
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const f16x8 codes = *reinterpret_cast<const f16x8*>(mem.v[buf][i][u][m] + lane * 16);
#pragma unroll
                    for (int j = 0; j < NP; ++j) acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(codes, p[j], acc[u], 0, 0, 0);
                }
            }
        }
    };

    if (from < to) {
        // while a step is worked on, the codes of the next one are turned into operands, those of
        // the one after it loaded, and its successor's blocks looked up; past the last step the same again
        auto next_of = [&](int t) { return t + 2 < to ? t + 2 : t; };
        Part<U> x;
        Scales now, then;
        int t1 = next_of(from), t2 = next_of(t1);
        x.load(a, pages(from), from, shift, h, wave, lane);
        uint32_t found = pages(t1);
        put(x, 0);
        now.set(a, x);
        x.load(a, found, t1, shift, h, wave, lane);
        found = pages(t2);
        int buf = 0;
        __syncthreads();
        for (int t = from; t < to; t += 2) {
            put(x, buf ^ 1);
            then.set(a, x);
            x.load(a, found, t2, shift, h, wave, lane);
            t2 = next_of(t2);
            found = pages(t2);
            compute(t, buf, now);
            now = then;
            buf ^= 1;
            __syncthreads();
        }
    }

    sum += __shfl_xor(sum, 32);
    if (k.parts > 1) {
        if (!real) return;
        float* ws = form_of<ROWS>(a).ws + ((uint64_t)k.slot * ROWS + 32 * wave + r) * (32 * U + 4);
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
    const float up = sum == 0.0f ? 0.0f : OUT / sum;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<four*>(&mem.rows[32 * wave + r][32 * u + 8 * j + 4 * hh]) =
                four{(T)(acc[u][4 * j] * up), (T)(acc[u][4 * j + 1] * up), (T)(acc[u][4 * j + 2] * up), (T)(acc[u][4 * j + 3] * up)};
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
