// What the forms of attention over the 8-bit cache share: how work is shared
// out, operands out of codes, the softmax's running state.
#pragma once

#include <type_traits>

#include "cache.hpp"

#if defined(__HIPCC__)
namespace lecb {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct AttendArgs {
    Seqs seqs;
    const void* q;
    void* out;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    float* ws;
    uint64_t q_token, q_head, out_token, out_head;
    uint32_t heads, group, dim;   // of the cache; query heads to each
    uint32_t window;              // 0: none
    int causal, fill;
    float scale;                  // times log2(e)
    uint32_t target;              // workgroups wished for
    uint32_t shortest;            // tiles that a part has at least
    uint32_t items;               // that the grid holds for each head
    uint32_t slots;               // that the workspace holds
};

// How the work is shared out.  A sequence's rows (tokens x query heads of one
// head of the cache) go by `rows` at a time, and the tiles that they see are
// split into parts of `part` tiles, chosen from all sequences' lengths so that
// about `target` workgroups share the whole evenly, whatever the lengths are:
// one long sequence among short ones is split further.  Numbers of items are
// bounded on the host by the same sums.  Parts of rows that are split leave their
// sums in slots of the workspace.
struct Item {
    uint32_t seq, rows_at, part, parts, slot, tiles;   // tiles: of each part
    uint32_t first_tile, last_tile;                    // of the sequence
};

struct Load {
    uint32_t first, tiles, rows;   // the tiles that the sequence's rows see, and how many rows by ROWS
};

template <int ROWS>
__device__ inline Load load_of(const AttendArgs& a, uint32_t s) {
    Load l = {0, 0, 0};
    if (s >= a.seqs.seqs) return l;
    const uint32_t n = a.seqs.count(s), len = a.seqs.length(s);
    if (n == 0) return l;
    l.rows = (uint32_t)(((uint64_t)n * a.group + ROWS - 1) / ROWS);
    if (a.seqs.bad(len) || len == 0) return l;
    const uint32_t at = len > n ? len - n : 0;
    l.first = a.window && at + 1 > a.window ? (at + 1 - a.window) / TILE_TOKENS : 0;
    l.tiles = (len + TILE_TOKENS - 1) / TILE_TOKENS - l.first;
    return l;
}

__device__ inline uint64_t sum64(uint64_t v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t lo = __shfl_xor((uint32_t)v, o), hi = __shfl_xor((uint32_t)(v >> 32), o);
        v += (uint64_t)hi << 32 | lo;
    }
    return v;
}
__device__ inline uint32_t scan32(uint32_t v, uint32_t lane) {   // of lanes 0 .. lane
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t b = __shfl_up(v, o);
        v += lane >= (uint32_t)o ? b : 0;
    }
    return v;
}

// Tiles of a part.
template <int ROWS>
__device__ inline uint32_t part_tiles(const AttendArgs& a, uint32_t lane) {
    uint64_t all = 0;
    for (uint32_t s0 = 0; s0 < a.seqs.seqs; s0 += 64) {
        const Load l = load_of<ROWS>(a, s0 + lane);
        all += (uint64_t)l.rows * l.tiles;
    }
    all = sum64(all) * a.heads;
    const uint64_t part = (all + a.target - 1) / a.target;
    return part > a.shortest ? part < 0x7fffffffu ? (uint32_t)part : 0x7fffffffu : a.shortest;
}

// The item numbered `w`, found by a wave; false: there are only `slot` of them.
template <int ROWS>
__device__ inline bool find_item(const AttendArgs& a, uint32_t w, uint32_t lane, Item& it) {
    const uint32_t part = part_tiles<ROWS>(a, lane);
    uint32_t items = 0, slots = 0;   // of the sequences before
    for (uint32_t s0 = 0; s0 < a.seqs.seqs; s0 += 64) {
        const Load l = load_of<ROWS>(a, s0 + lane);
        const uint32_t parts = l.tiles > part ? (l.tiles + part - 1) / part : 1;
        const uint32_t mine = l.rows * parts, split = parts > 1 ? mine : 0;
        const uint32_t upto = scan32(mine, lane) + items, slots_upto = scan32(split, lane) + slots;
        const uint64_t hit = __ballot(w < upto);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const uint32_t k = w - __shfl(upto - mine, at);
            it.seq = s0 + at;
            it.parts = __shfl(parts, at);
            it.rows_at = k / it.parts;
            it.part = k % it.parts;
            it.slot = __shfl(slots_upto - split, at) + k;
            it.tiles = part;
            it.first_tile = __shfl(l.first, at);
            it.last_tile = it.first_tile + __shfl(l.tiles, at);
            return true;
        }
        items = __shfl(upto, 63);
        slots = __shfl(slots_upto, 63);
    }
    it.slot = items;
    return false;
}

// Rows of no sequence, by the workgroups that have no item.
template <typename T>
__device__ inline void fill_rows(const AttendArgs& a, uint32_t me, uint32_t all) {
    uint32_t second = 0;
    const uint32_t n = a.seqs.outside(&second), b = n ? a.seqs.begin(0) : 0;
    const uint32_t width = a.heads * a.group;
    for (uint32_t i = me; i < n; i += all) {
        T* row = reinterpret_cast<T*>(a.out) + (uint64_t)(i < b ? i : second + i - b) * a.out_token;
        for (uint32_t h = 0; h < width; ++h)
            for (uint32_t d = threadIdx.x; d < a.dim; d += blockDim.x) row[h * a.out_head + d] = (T)0.0f;
    }
}

// Four codes as halves, exact: a byte q + 128 under 0x64 is the half 1024 + 128 + q.
__device__ inline void halves(uint32_t codes, uint32_t* out) {
    const uint32_t u = codes ^ 0x80808080u;
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w = __builtin_amdgcn_perm(0x64646464u, u, i ? 0x04030402u : 0x04010400u);
        out[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, w) - off);
    }
}
__device__ inline f16x8 operand(uint32_t lo, uint32_t hi) {
    u32x4 w;
    uint32_t h[4];
    halves(lo, h);
    halves(hi, h + 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = h[i];
    return __builtin_bit_cast(f16x8, w);
}

// A row of q as halves: times the power of two that takes its largest element
// to 2^14 .. 2^15 (its numbers down to 2^-29 of that are exact then; fp16 stays
// as it is), and in three parts where it has 24 bits.  The softmax's weights go
// in one part of 11 bits where results have 8, else in two.
template <typename T>
struct Parts;
template <>
struct Parts<__bf16> {
    static constexpr int Q = 1, P = 1;
    static constexpr bool LIFT = true;
};
template <>
struct Parts<_Float16> {
    static constexpr int Q = 1, P = 2;
    static constexpr bool LIFT = false;
};
template <>
struct Parts<float> {
    static constexpr int Q = 3, P = 2;
    static constexpr bool LIFT = true;
};

// The running state of a row's softmax, in units that make it last: weights are
// p = 2^(x + ref), x the score times log2(e), and ref = 30 - max(x + e) where
// 2^e is the power of two just above the scale of x's values (e >= -60).  So p
// times that scale, what the second product takes, is at most 2^30 whatever the
// scales are (2^15 as a half, OUT undoes the rest), with 40 bits below it before
// halves run out, and p itself stays within 2^90 and 2^-98.
constexpr float REF_TOP = 30.0f;
constexpr float P_DOWN = 0x1p-15f;   // into halves
constexpr float OUT = 0x1p15f;       // and back
constexpr int SCALE_LOW = -60;

__device__ inline float scale_exponent(float s) {
    // 0, infinities and NaN give 0 or what they stand for below; all that counts is that p stays finite
    const int e = __builtin_amdgcn_frexp_expf(s);
    return (float)(s == 0.0f ? SCALE_LOW : e > SCALE_LOW ? e : SCALE_LOW);
}
__device__ inline float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float inf() { return __uint_as_float(0x7f800000u); }

}  // namespace lecb
#endif
