// Attention over the 8-bit cache: the form for few rows (decoding steps).
#pragma once

#include "attend.hpp"

#if defined(__HIPCC__)
namespace lecb {

// Few rows: a workgroup takes 16 rows of one head over a part of the tiles,
// its waves tile by tile in turn, each with a softmax of its own; their sums are
// joined at the end.  Matrix instructions by 16 x 16 x 32, transposed: codes of
// 16 tokens (then of 16 dimensions of the values) times the rows, so that a row's
// scores stand in one lane of each 16, four tokens each, and are the second
// product's operand as they are; values are stored in that order of tokens.
// Neither codes nor scores go through LDS.
//
// Bound by HBM, with vector instructions (codes to halves, 1.25 a code) at half
// of their rate: 64 sequences of up to 8192 tokens, 32 heads to 8 of 128
// dimensions, 96 us, 5.6 TB/s of codes; one token after 262144 88 us, 6.1 TB/s.  With two sets of
// registers for codes (a whole tile ahead, 3 waves a SIMD instead of 4) these took 104
// and 92.  Eight waves a workgroup: 104 -> 111 and 95 -> 93 with all launches.  A call
// of few tokens lasts as long as its chain of loads (lengths, blocks, codes): 6.7 us
// for 1000 tokens and 2.7 of attend_join_kernel's.
template <typename T, int U, int WAVES>
struct FewMemory {
    union {
        T q[FEW_ROWS][32 * U];
        float sum[WAVES][FEW_ROWS][68];
    };
    float ref[WAVES][FEW_ROWS], l[WAVES][FEW_ROWS];
};

template <typename T, int U, int WAVES>
__device__ inline void attend_few(const AttendArgs& a, const Item& it, uint32_t h, FewMemory<T, U, WAVES>& mem) {
    // weights in two parts, 22 bits, for every type: the second products are not what bounds this form
    constexpr int ROWS = FEW_ROWS, NQ = Parts<T>::Q, NP = 2, THREADS = 64 * WAVES;
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    Work k;
    if (!work_of<ROWS>(a, it, h, k)) return;
    if (k.bad) {
        bad_rows<T>(a, k, h);
        return;
    }
    const uint32_t seq = it.seq, shift = __builtin_ctz(a.seqs.block / TILE_TOKENS);
    const int from = k.from, to = k.to, lo_most = k.lo_most, hi_least = k.hi_least;

    // a tile's codes as they lie and, in even and odd lanes, the scales of its keys and values
    u32x4 kc[U], vc[U];
    float scales = 0.0f;
    bool none = false, none_next = false;   // the table names no block of the cache
    auto page = [&](int t) { return a.seqs.page(seq, (uint32_t)t >> shift); };
    auto cell_of = [&](uint32_t found) {
        const uint32_t page = uniform(found);
        none_next = page >= a.seqs.blocks;
        return (uint64_t)(none_next ? 0 : page) * a.heads + h;
    };
    auto place = [&](uint64_t cell, int t) {
        return ((cell << shift) + ((uint32_t)t & ((1u << shift) - 1))) * (U * UNIT_BYTES) + lane * 16;
    };
    auto load_codes = [&](const uint8_t* codes, uint64_t at, u32x4 (&w)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) w[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes + at + u * UNIT_BYTES));
    };
    auto load_scales = [&](uint64_t cell) { return (lane & 1 ? a.v_scale : a.k_scale)[cell]; };
    auto next_of = [&](int t) { return t + WAVES < to ? t + WAVES : t; };

    // the first tile is on its way while the rows are made ready
    int t = from + (int)wave;
    uint32_t found = 0;
    if (t < to) {
        const uint32_t first = page(t);
        found = page(next_of(t));
        const uint64_t cell = cell_of(first), at = place(cell, t);
        none = none_next;
        load_codes(a.k, at, kc);
        load_codes(a.v, at, vc);
        scales = load_scales(cell);
    }
    stage_rows(a, k, h, ROWS, 32 * U, &mem.q[0][0]);
    __syncthreads();

    // rows: lane r of each 16 has row r, dimensions 32 u + 8 g and on
    const uint32_t row = k.r0 + r;
    f16x8 q[U][NQ];
    const Factor factor = load_row<T, U, 16>(a, mem.q[r], 8 * g, 32, q);
    const int pos = k.old + (row < k.rows ? (int)(row / a.group) : 0);
    const int hi = a.causal ? pos : k.len - 1, lo = a.window ? pos - (int)a.window + 1 : 0;

    f32x4 acc[2 * U];
    float ref = inf(), sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Codes have one set of registers: the next tile's keys are asked for once this one's are
    // operands, its values after theirs, its block one tile ahead.  Past the last tile the
    // same one is loaded again.
    for (; t < to; t += WAVES) {
        const int t1 = next_of(t), at = t * (int)TILE_TOKENS;
        const float ks = key_scale(of_lane(scales, 0), !none), vs = of_lane(scales, 1);
        f32x4 s[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const f16x8 codes = operand(kc[u][2 * b], kc[u][2 * b + 1]);
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes, q[u][j], s[b], 0, 0, 0);
            }
        const uint64_t cell = cell_of(found), next_at = place(cell, t1);
        load_codes(a.k, next_at, kc);
        scales = load_scales(cell);
        none = none_next;
        found = page(next_of(t1));

        // all rows see all of the tile's tokens, and the larger product is the larger score
        const bool plain = at >= lo_most && at + (int)TILE_TOKENS - 1 <= hi_least && a.scale >= 0.0f && ks >= 0.0f;
        const bool number = finite(vs);
        const float down = number ? vs * P_DOWN : 0.0f, unit = scale_exponent(vs);
        float f = factor.times(ks), v[8], most = -inf();
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s[i / 4][i % 4];
        if (!plain) {
            asm volatile("");   // not to be done and then selected from
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int token = at + 4 * (int)g + i % 4 + i / 4 * 16;
                v[i] = token <= hi && token >= lo ? v[i] * f : -inf();
            }
            f = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, v[i]);
        most = max_of_quarters(most * f);
        // values without a number to scale them: no number to the rows that see one of them
        if (!number && most != -inf()) sum = __uint_as_float(0x7fc00000u);
        const float next = REF_TOP - (most + unit);
        if (__ballot(next < ref - LAG)) {
            const float root = next < ref ? root_of(next - ref) : 1.0f, down_by = root * root;
            sum = sum * root * root;
#pragma unroll
            for (int i = 0; i < 2 * U; ++i) acc[i] *= down_by;
            ref = fminf(ref, next);
        }
        const float base = ref == inf() ? 0.0f : ref;
        f16x8 p[NP];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = exp2_of(fmaf(v[i], f, base));
            sum += v[i];
            v[i] = product(v[i], down);
        }
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[j][i] = (_Float16)v[i];
                v[i] -= (float)p[j][i];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const f16x8 codes = operand(vc[u][2 * b], vc[u][2 * b + 1]);
#pragma unroll
                for (int j = 0; j < NP; ++j)
                    acc[2 * u + b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes, p[j], acc[2 * u + b], 0, 0, 0);
            }
        load_codes(a.v, next_at, vc);
    }
    __syncthreads();   // the rows in LDS are no longer needed

    // the waves' sums, joined in their order
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (g == 0) {
        mem.ref[wave][r] = ref;
        mem.l[wave][r] = sum;
    }
    __syncthreads();
    float lowest = mem.ref[0][r];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) lowest = fminf(lowest, mem.ref[i][r]);
    const float down_by = ref == lowest ? 1.0f : exp2_of(lowest - ref);
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) acc[i] *= down_by;
    float* ws = form_of<ROWS>(a).ws + (uint64_t)k.slot * ROWS * (32 * U + 4);
#pragma unroll
    for (int d0 = 0; d0 < U; d0 += 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * d0 + i < 2 * U) *reinterpret_cast<f32x4*>(&mem.sum[wave][r][16 * i + 4 * g]) = acc[2 * d0 + i];
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < ROWS * 16; i += THREADS) {
            const uint32_t row = i / 16, d = i % 16 * 4, at = 32 * d0 + d;
            if (row >= k.have || at >= 32 * U) continue;
            f32x4 v = *reinterpret_cast<const f32x4*>(&mem.sum[0][row][d]);
#pragma unroll
            for (int j = 1; j < WAVES; ++j) v += *reinterpret_cast<const f32x4*>(&mem.sum[j][row][d]);
            float least = mem.ref[0][row], l = 0.0f;
#pragma unroll
            for (int j = 1; j < WAVES; ++j) least = fminf(least, mem.ref[j][row]);
#pragma unroll
            for (int j = 0; j < WAVES; ++j) {
                const float root = mem.ref[j][row] == least ? 1.0f : root_of(least - mem.ref[j][row]);
                l += mem.l[j][row] * root * root;
            }
            if (k.parts > 1) {
                *reinterpret_cast<f32x4*>(ws + row * (32 * U + 4) + 4 + at) = v;
                if (at == 0) {
                    ws[row * (32 * U + 4)] = least;
                    ws[row * (32 * U + 4) + 1] = l;
                }
            } else {
                const float up = l == 0.0f ? 0.0f : OUT / l;
                const T o[4] = {(T)(v[0] * up), (T)(v[1] * up), (T)(v[2] * up), (T)(v[3] * up)};
                put_four(a, k, h, k.r0 + row, at, o);
            }
        }
        __syncthreads();
    }
}

}  // namespace lecb
#endif
