// What the forms of attention over the 8-bit cache share: how work is shared
// out, operands out of codes, the softmax's running state.
#pragma once

#include <type_traits>

#include "cache.hpp"

#if defined(__HIPCC__)
namespace lecb {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline uint32_t of_lane(uint32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ inline float of_lane(float v, int lane) { return __uint_as_float(of_lane(__float_as_uint(v), lane)); }

constexpr int FEW_ROWS = 16;   // of a workgroup in the form for few rows; in that for many 128 or 256

// How one form's work is shared out.  A sequence's rows (tokens x query heads of
// one head of the cache) go by ROWS at a time, and the tiles that they see are
// split into parts of one length, chosen from all sequences' lengths so that
// about `target` workgroups share the whole evenly, whatever the lengths are:
// one long sequence among short ones is split further.  Numbers of items are
// bounded on the host by the same sums.  Parts of rows that are split leave their
// sums in slots of the workspace.
struct Form {
    float* ws;
    uint32_t target;     // workgroups wished for
    uint32_t shortest;   // tiles that a part has at least
    uint32_t slots;      // that the workspace holds, for all heads
};

struct AttendArgs {
    Seqs seqs;
    const void* q;
    void* out;
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    uint64_t q_token, q_head, out_token, out_head;
    uint32_t heads, group, dim;   // of the cache; query heads to each
    uint32_t window;              // 0: none
    int causal, fill;
    float scale;                  // times log2(e)
    uint32_t few;                 // rows of a sequence up to which the form for few takes it
    Form form[2];                 // few, many
};

struct Item {
    uint32_t seq, rows_at, part, parts, slot, tiles;   // tiles: of each part
    uint32_t first_tile, last_tile;                    // of the sequence
    uint32_t begin, n, len;                            // its rows, and its tokens with them
};

struct Load {
    uint32_t first, tiles, rows;   // the tiles that the sequence's rows see, and how many rows by ROWS
    uint32_t begin, n, len;        // as in Item
};

template <int ROWS>
__device__ inline const Form& form_of(const AttendArgs& a) {
    return a.form[ROWS != FEW_ROWS];
}

template <int ROWS>
__device__ inline Load load_of(const AttendArgs& a, uint32_t s) {
    Load l = {};
    if (s >= a.seqs.seqs) return l;
    const uint32_t n = a.seqs.count(s), len = a.seqs.length(s);
    l.begin = a.seqs.begin(s);
    l.n = n;
    l.len = len;
    if (n == 0 || (n * a.group > a.few) != (ROWS != FEW_ROWS)) return l;   // the other form's
    l.rows = (n * a.group + ROWS - 1) / ROWS;
    if (a.seqs.bad(len) || len == 0) return l;
    const uint32_t at = len > n ? len - n : 0;
    l.first = a.window && at + 1 > a.window ? (at + 1 - a.window) / TILE_TOKENS & ~1u : 0;
    l.tiles = (len + TILE_TOKENS - 1) / TILE_TOKENS - l.first;
    return l;
}

// Over lanes 0 .. limit - 1 (a power of two), the others holding zeros.
__device__ inline uint64_t sum64(uint64_t v, uint32_t limit) {
    for (uint32_t o = 1; o < limit; o <<= 1) {
        const uint32_t lo = __shfl_xor((uint32_t)v, o), hi = __shfl_xor((uint32_t)(v >> 32), o);
        v += (uint64_t)hi << 32 | lo;
    }
    return (uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v);
}
// For lane i the sum of lanes 0 .. i.
__device__ inline uint32_t scan32(uint32_t v, uint32_t lane, uint32_t limit) {
    for (uint32_t o = 1; o < limit; o <<= 1) {
        const uint32_t b = __shfl_up(v, o);
        v += lane >= o ? b : 0;
    }
    return v;
}

// The item numbered `w`, found by a wave; false: there are only `slot` of them.
// With JOIN items are whole rows that were split.  Parts have an even number of tiles.
template <int ROWS, bool JOIN>
__device__ inline bool find_item(const AttendArgs& a, uint32_t w, uint32_t lane, Item& it) {
    const Form& f = form_of<ROWS>(a);
    const Load first = load_of<ROWS>(a, lane);   // of the first 64 sequences, all of them in most calls
    uint64_t all = (uint64_t)first.rows * first.tiles;
    for (uint32_t s0 = 64; s0 < a.seqs.seqs; s0 += 64) {
        const Load l = load_of<ROWS>(a, s0 + lane);
        all += (uint64_t)l.rows * l.tiles;
    }
    uint32_t limit = 1;   // lanes that hold something
    while (limit < 64 && limit < a.seqs.seqs) limit *= 2;
    all = sum64(all, limit) * a.heads + f.target - 1;
    const uint64_t wish = (all >> 32 ? all / f.target : (uint32_t)all / f.target) + 1 & ~1ull;
    const uint32_t part = uniform(wish > f.shortest ? wish < 0x7ffffffeu ? (uint32_t)wish : 0x7ffffffeu : f.shortest);
    uint32_t items = 0, slots = 0;   // of the sequences before
    for (uint32_t s0 = 0; s0 < a.seqs.seqs; s0 += 64) {
        const Load l = s0 == 0 ? first : load_of<ROWS>(a, s0 + lane);
        const uint32_t parts = l.tiles > part ? (l.tiles + part - 1) / part : 1;
        const uint32_t split = parts > 1 ? l.rows * parts : 0;
        const uint32_t mine = JOIN ? parts > 1 ? l.rows : 0 : l.rows * parts;
        const uint32_t upto = scan32(mine, lane, limit) + items, slots_upto = scan32(split, lane, limit) + slots;
        const uint64_t hit = __ballot(w < upto);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const uint32_t k = w - of_lane(upto - mine, at);
            it.seq = uniform(s0 + at);
            it.parts = of_lane(parts, at);
            const uint32_t each = JOIN ? 1 : it.parts;
            it.rows_at = of_lane(l.rows, at) - 1 - k / each;   // the rows that see most come first
            it.part = k % each;
            it.slot = of_lane(slots_upto - split, at) + it.rows_at * it.parts + it.part;
            it.tiles = part;
            it.first_tile = of_lane(l.first, at);
            it.last_tile = it.first_tile + of_lane(l.tiles, at);
            it.begin = of_lane(l.begin, at);
            it.n = of_lane(l.n, at);
            it.len = of_lane(l.len, at);
            return true;
        }
        items = of_lane(upto, limit - 1);
        slots = of_lane(slots_upto, limit - 1);
    }
    it.slot = items;
    return false;
}

// What a workgroup of either form works on: rows, and the tiles that they see.
struct Work {
    uint32_t begin, rows, r0, have, slot, parts;   // the sequence's first row and their number; of this item
    int old, len;                                  // tokens before the sequence's rows, and with them
    int from, to;                                  // tiles
    int hi_least, lo_most;                         // whole ones are seen by every row
    bool bad;
};

template <int ROWS>
__device__ inline bool work_of(const AttendArgs& a, const Item& it, uint32_t h, Work& k) {
    const uint32_t n = it.n, len = it.len;
    k.begin = it.begin;
    k.rows = n * a.group;
    k.slot = it.slot * a.heads + h;
    k.parts = it.parts;
    // starts that do not rise make more of either than there is room for
    if (it.rows_at >= (k.rows + ROWS - 1) / ROWS || (it.parts > 1 && k.slot >= form_of<ROWS>(a).slots)) return false;
    k.r0 = it.rows_at * ROWS;
    k.have = k.rows - k.r0 < (uint32_t)ROWS ? k.rows - k.r0 : ROWS;
    k.bad = a.seqs.bad(len);
    k.len = (int)len;
    k.old = (int)len - (int)n;
    const int first = (int)(k.r0 / a.group), last = (int)((k.r0 + k.have - 1) / a.group), w = (int)a.window;
    const int hi_most = a.causal ? k.old + last : k.len - 1, lo_least = w ? k.old + first - w + 1 : 0;
    k.hi_least = a.causal ? k.old + first : k.len - 1;
    k.lo_most = w ? k.old + last - w + 1 : 0;
    const uint64_t at = (uint64_t)it.first_tile + (uint64_t)it.part * it.tiles;
    k.from = (int)at;
    k.to = (int)it.last_tile;
    if (at + it.tiles < (uint64_t)k.to) k.to = (int)(at + it.tiles);
    if (lo_least > 0 && lo_least / (int)TILE_TOKENS > k.from) k.from = lo_least / (int)TILE_TOKENS & ~1;
    const int seen = hi_most < 0 ? 0 : hi_most / (int)TILE_TOKENS + 1;
    if (seen < k.to) k.to = seen;
    return true;
}

// The rows of a sequence that does not fit its row of the table.
template <typename T>
__device__ inline void bad_rows(const AttendArgs& a, const Work& k, uint32_t h) {
    for (uint32_t i = 0; i < k.have; ++i) {
        const uint32_t row = k.r0 + i;
        T* o = reinterpret_cast<T*>(a.out) + (uint64_t)(k.begin + row / a.group) * a.out_token +
               (uint64_t)(h * a.group + row % a.group) * a.out_head;
        for (uint32_t d = threadIdx.x; d < a.dim; d += blockDim.x) o[d] = (T)__uint_as_float(0x7fc00000u);
    }
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
// in two parts of 11 bits each; in the form for many rows in one where results have 8 bits: a second
// part costs it a third (two prompts of up to 4096 tokens 276 -> 357 us, 512 after 32256 301 -> 410), and one leaves
// 9 of 100 results of 8 bits on the other side of their rounding, their error 1 % larger.  The form for few
// takes it along: 64 sequences of up to 8192 tokens 102.6 -> 103.4 us, one token after 262144 93.3 -> 92.9.
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
// 2^e is the power of two just above the scale of x's values, -60 <= e <= 128.  ref
// follows a larger maximum only once it is LAG behind, as sums have to be scaled
// whenever it moves: in a prompt of 4096 tokens after nearly each pair of tiles
// without that, once or twice with it.  So p times that scale, what the second
// product takes, is at most 2^34, with 36 bits below a largest of 2^30 before halves
// run out; scales below 2^-60 lose as many of these as they are below it.  p itself is
// at most 2^94, and the one that ref was taken from 2^-98 or more: beside the largest
// scale there can be, the sum of weights has 28 bits left in the exponential's range
// below that one, and one more for each bit that the scale is smaller.
constexpr float REF_TOP = 30.0f, LAG = 4.0f;
constexpr float P_DOWN = 0x1p-19f;   // into halves: at most 2^(30 + LAG - 19)
constexpr float P_DOWN_LOG2 = -19.0f;
constexpr float OUT = 0x1p19f;       // and back
constexpr int SCALE_LOW = -60;

__device__ inline float scale_exponent(float s) {
    // infinities and NaN give 0, as all that counts is that p stays finite; zero the lowest, to stand behind all others
    const int e = __builtin_amdgcn_frexp_expf(s);
    return (float)(s == 0.0f ? SCALE_LOW : e > SCALE_LOW ? e : SCALE_LOW);
}
// a * b rounded to 32 bits before it is split: the compiler would fuse the product with the
// first part's conversion, which now and then rounds the other way than what the second part is the rest of.
__device__ inline float product(float a, float b) {
    float p = a * b;
    asm("" : "+v"(p));
    return p;
}
__device__ inline float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
// What takes sums of weights to a reference that is d (<= 0) away, as the root of it: multiplied in twice.  References lie
// up to 2^188 apart where the scales do, further than one factor reaches, and sums of weights up to 2^94 each still count then.
__device__ inline float root_of(float d) { return exp2_of(0.5f * d); }
// The largest of the lanes 32 apart, and of those 16 apart.
__device__ inline float max_of_halves(float v) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ inline float max_of_quarters(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return max_of_halves(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
}
__device__ inline float inf() { return __uint_as_float(0x7f800000u); }
// Whether s is neither infinite nor NaN, in scalar registers where s is (attend_few has none of the others to spare).
__device__ inline bool finite(float s) { return __float_as_uint(s) << 1 < 0xff000000u; }

// A block's scale of keys; NaN where it is no number or there is no such block: an infinite one would leave tokens
// whose products are negative out of the softmax, which their keys, infinities and 0 times infinity, are not.
__device__ inline float key_scale(float s, bool there) {
    return there && (__float_as_uint(s) & 0x7fffffffu) < 0x7f800000u ? s : __uint_as_float(0x7fc00000u);
}

// Rows of q into LDS, `pitch` elements apart, zeros past the head's dimensions and
// past the last row: what all waves of a workgroup then take their operands from.
template <typename T>
__device__ inline void stage_rows(const AttendArgs& a, const Work& k, uint32_t h, uint32_t rows, uint32_t pitch, T* to) {
    typedef T piece __attribute__((ext_vector_type(16 / sizeof(T))));
    typedef piece loose __attribute__((aligned(sizeof(T))));
    constexpr uint32_t N = 16 / sizeof(T);
    const uint32_t across = pitch / N;
#pragma unroll 2
    for (uint32_t i = threadIdx.x; i < rows * across; i += blockDim.x) {
        const uint32_t row = k.r0 + i / across, d = i % across * N;
        const T* p = reinterpret_cast<const T*>(a.q) + (uint64_t)(k.begin + row / a.group) * a.q_token +
                     (uint64_t)(h * a.group + row % a.group) * a.q_head + d;
        piece x = {};
        if (row < k.rows && d < a.dim) {
            if (d + N <= a.dim) {
                x = *reinterpret_cast<const loose*>(p);
            } else {
#pragma unroll
                for (uint32_t e = 0; e < N; ++e)
                    if (d + e < a.dim) x[e] = p[e];
            }
        }
        *reinterpret_cast<piece*>(to + i * N) = x;
    }
}

// What takes a row's products of codes to scores, with the block's scale: its power of two, to 2^-163, comes in two halves,
// so that small queries and large keys, or the other way round, meet within the range of 32 bits and lose nothing.
struct Factor {
    float a, b;
    __device__ float times(float scale) const { return a * scale * b; }
};

// One row as operands: N pieces of eight dimensions, d0 + step i and on; the lanes
// that share a row are LANES apart.
template <typename T, int N, int LANES>
__device__ inline Factor load_row(const AttendArgs& a, const T* row, uint32_t d0, uint32_t step, f16x8 (&q)[N][Parts<T>::Q]) {
    typedef T piece __attribute__((ext_vector_type(8)));
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const piece x = *reinterpret_cast<const piece*>(row + step * u + d0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint((float)x[e]) & 0x7fffffffu;
            top = b > top ? b : top;
        }
    }
#pragma unroll
    for (int o = LANES; o < 64; o <<= 1) {
        const uint32_t b = __shfl_xor(top, o);
        top = b > top ? b : top;
    }
    int lift = 0;
    if (Parts<T>::LIFT && top != 0) lift = 15 - __builtin_amdgcn_frexp_expf(__uint_as_float(top));
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const piece x = *reinterpret_cast<const piece*>(row + step * u + d0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f = Parts<T>::LIFT ? ldexpf((float)x[e], lift) : (float)x[e];
#pragma unroll
            for (int j = 0; j < Parts<T>::Q; ++j) {
                q[u][j][e] = (_Float16)f;
                f -= (float)q[u][j][e];
            }
        }
    }
    const int half = lift / 2;
    return {top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : ldexpf(a.scale, -half), ldexpf(1.0f, half - lift)};
}

// Four neighbouring results, as far as the head's dimensions go.
template <typename T>
__device__ inline void put_four(const AttendArgs& a, const Work& k, uint32_t h, uint32_t row, uint32_t d, const T (&v)[4]) {
    typedef T four __attribute__((ext_vector_type(4)));
    typedef four loose __attribute__((aligned(sizeof(T))));
    T* o = reinterpret_cast<T*>(a.out) + (uint64_t)(k.begin + row / a.group) * a.out_token +
           (uint64_t)(h * a.group + row % a.group) * a.out_head + d;
    if (d + 4 <= a.dim) {
        *reinterpret_cast<loose*>(o) = four{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (uint32_t e = 0; e < 3; ++e)
            if (d + e < a.dim) o[e] = v[e];
    }
}

}  // namespace lecb
#endif
