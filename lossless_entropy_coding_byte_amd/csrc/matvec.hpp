// What the products with 4-bit weights share: matrix instructions' operands out
// of codes and tokens, loads of tokens, the last rounding.
#pragma once

#include "layers.hpp"

namespace lecb {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Operands of the matrix instructions for tokens of type X, and their product.
//
// An instruction takes 32 columns (64 for bytes in pairs of words): of a token
// (first operand) and of a row of W (second), eight of them from each lane in
// any order that both sides share.
//
// bytes: a code's four bits as the upper half of a byte, 16 q, the even
// columns and the odd ones in a register each.
//
// 16 bits: a code's four bits, the sign's turned over, as the upper bits of the
// mantissa of 2^-8: 2^-8 (1 + (q + 8) / 16), exactly, for one logic operation a
// pair of codes (columns p and p + 4) after one shift; a conversion to float
// and a packing take four times as long.  What is too much, 1.5 2^-8 times the
// group's sum of x, is put into the sum beforehand: by an instruction whose
// second operand is EXCESS, or from sums made before (Tokens).  2^-8 keeps the
// sum over a group within the range of x, exact for its smallest numbers too.
// SCALE, of a group's scale, undoes 16 and 2^-8; FACTOR, of the result, 16.
template <typename X>
struct Operand;

// Pairs of halves (p, p + 4), p = 0..3, out of eight halves in order.
__device__ inline u32x4 pairs_of_halves(u32x4 x) {
    return {__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
            __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

template <>
struct Operand<__bf16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float SCALE = 4096.0f, FACTOR = 1.0f;
    static constexpr bool OFFSET = true;
    static constexpr uint32_t EXCESS = 0xBBC0BBC0u;   // -1.5 2^-8, twice
    static __device__ A weights(uint32_t w) {
        return {((w << 3) & 0x00780078u) ^ 0x3BC03BC0u, ((w >> 1) & 0x00780078u) ^ 0x3BC03BC0u,
                ((w >> 5) & 0x00780078u) ^ 0x3BC03BC0u, ((w >> 9) & 0x00780078u) ^ 0x3BC03BC0u};
    }
    static __device__ u32x4 order(u32x4 x) { return pairs_of_halves(x); }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {   // 32 tokens, 32 rows, 16 columns
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ float dot(uint32_t a, uint32_t b, float c) {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
    }
};
template <>
struct Operand<_Float16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float SCALE = 4096.0f, FACTOR = 1.0f;
    static constexpr bool OFFSET = true;
    static constexpr uint32_t EXCESS = 0x9E009E00u;
    static __device__ A weights(uint32_t w) {
        return {((w << 6) & 0x03C003C0u) ^ 0x1E001E00u, ((w << 2) & 0x03C003C0u) ^ 0x1E001E00u,
                ((w >> 2) & 0x03C003C0u) ^ 0x1E001E00u, ((w >> 6) & 0x03C003C0u) ^ 0x1E001E00u};
    }
    static __device__ u32x4 order(u32x4 x) { return pairs_of_halves(x); }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
    static __device__ f32x16 mul32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    }
    static __device__ float dot(uint32_t a, uint32_t b, float c) {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
    }
};
template <>
struct Operand<int8_t> {
    typedef u32x2 A;
    typedef i32x4 Acc;
    static constexpr float SCALE = 1.0f, FACTOR = 0.0625f;
    static constexpr bool OFFSET = false;
    static __device__ A weights(uint32_t w) { return {(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u}; }
    static __device__ u32x2 order(u32x2 x) {
        return {__builtin_amdgcn_perm(x.y, x.x, 0x06040200u), __builtin_amdgcn_perm(x.y, x.x, 0x07050301u)};
    }
    static __device__ u32x4 order(u32x4 x) {   // two times eight bytes
        const u32x2 a = order(u32x2{x.x, x.y}), b = order(u32x2{x.z, x.w});
        return {a.x, a.y, b.x, b.y};
    }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0,
                                                     0, 0);
    }
    // two words at once: 64 columns an instruction, at twice the rate
    static __device__ Acc mul2(u32x4 a, A b0, A b1, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                     i32x4{(int)b0.x, (int)b0.y, (int)b1.x, (int)b1.y}, c, 0, 0, 0);
    }
    static __device__ i32x16 mul32(A a, A b, i32x16 c) {
        return __builtin_amdgcn_mfma_i32_32x32x16_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0,
                                                     0);
    }
    static __device__ i32x16 mul32x2(u32x4 a, A b0, A b1, i32x16 c) {   // 32 columns
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                     i32x4{(int)b0.x, (int)b0.y, (int)b1.x, (int)b1.y}, c, 0, 0, 0);
    }
};

// Eight neighbouring entries of a token's tile (8 sizeof(X) bytes), in order;
// of the first `left` (at least one) columns only, zeros after them: entries
// past them repeat the last one's load, so that all are in flight at once.
template <typename X>
__device__ inline typename Operand<X>::A load_eight(const X* tile, uint32_t col) {
    typedef typename Operand<X>::A any __attribute__((aligned(sizeof(X))));
    return *reinterpret_cast<const any*>(tile + col);
}
template <typename X>
__device__ inline typename Operand<X>::A load_eight(const X* tile, uint32_t col, uint32_t left) {
    constexpr int PER = 4 / sizeof(X), BITS = 8 * sizeof(X);
    typename Operand<X>::A v{};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t at = col + i < left ? col + i : left - 1;
        const uint32_t e = sizeof(X) == 1 ? reinterpret_cast<const uint8_t*>(tile)[at]
                                          : reinterpret_cast<const uint16_t*>(tile)[at];
        v[i / PER] |= (col + i < left ? e : 0u) << (BITS * (i % PER));
    }
    return v;
}

// A token's 128 columns of a tile as 16-byte units, each what a lane gives one
// instruction of 16 bits or of 64 columns of bytes: 16 bits, unit u holds
// columns 8 u ..; bytes, unit 4 p + c holds columns 64 p + 8 c .. and 64 p + 32
// + 8 c ...  So lane 16 c + r takes units 4 p + c of token r, p < PIECES.
template <typename X>
struct Tokens {
    static constexpr int PIECES = 2 * sizeof(X), UNITS = 4 * PIECES;
    static __device__ uint32_t column(uint32_t unit) {
        return sizeof(X) == 1 ? 64 * (unit >> 2) + 8 * (unit & 3) : 8 * unit;
    }
    static __device__ u32x4 load(const X* tile, uint32_t unit) {
        if constexpr (sizeof(X) == 1)
            return join(load_eight(tile, column(unit)), load_eight(tile, column(unit) + 32));
        else
            return load_eight(tile, column(unit));
    }
    static __device__ u32x4 load(const X* tile, uint32_t unit, uint32_t left) {
        if constexpr (sizeof(X) == 1)
            return join(load_eight(tile, column(unit), left), load_eight(tile, column(unit) + 32, left));
        else
            return load_eight(tile, column(unit), left);
    }
    static __device__ u32x4 join(u32x2 a, u32x2 b) { return {a.x, a.y, b.x, b.y}; }
};

struct MatvecArgs {
    const void* x;
    const float* xscale;
    const u32x4* tiles;
    const void* scales;
    void* y;
    void* ws;
    uint64_t x_stride, y_stride, n, k, m;
    uint32_t nt, kt;
    int xscale_stride, y_type;
    uint32_t splits;   // shares of the columns over workgroups; above 1, sums go to `parts`
    float* parts;      // [splits][m][16 nt]
};

// The last step of a sum: the token's factor, one rounding, four outputs.
__device__ inline void store_y(const MatvecArgs& a, uint64_t token, uint64_t col, f32x4 v) {
    const uint64_t at = token * a.y_stride + col, left = a.n - col;
    if (a.xscale) v *= a.xscale[a.xscale_stride ? token : 0];
    if (left >= 4) {
        if (a.y_type == LECB_F32) {
            typedef f32x4 loose __attribute__((aligned(4)));
            *reinterpret_cast<loose*>(reinterpret_cast<float*>(a.y) + at) = v;
        } else if (a.y_type == LECB_BF16) {
            typedef bf16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<__bf16*>(a.y) + at) =
                bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
            typedef f16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<_Float16*>(a.y) + at) =
                f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 3; ++e) {
        if ((uint64_t)e >= left) continue;
        if (a.y_type == LECB_F32)
            reinterpret_cast<float*>(a.y)[at + e] = v[e];
        else if (a.y_type == LECB_BF16)
            reinterpret_cast<__bf16*>(a.y)[at + e] = (__bf16)v[e];
        else
            reinterpret_cast<_Float16*>(a.y)[at + e] = (_Float16)v[e];
    }
}

// Waits for this wave's LDS accesses and then for the other waves.  Loads from
// memory stay in flight, those on their way to LDS too.
__device__ inline void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// BYTES (4 or 16) from `from` (the same in every lane) plus each lane's offset
// straight to LDS, lane after lane from `to` on; there after loads_done and, for
// the other waves, a barrier.  The buffer form: after a global one the compiler
// waits for everything in flight at the next load it needs.
template <int BYTES>
__device__ inline void load_to_lds(const void* from, uint32_t offset, void* to) {
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(from), 0, 0xffffffffu, 0x00020000);
    typedef __attribute__((address_space(3))) void* Lds;
    if constexpr (BYTES == 16)   // the builtin takes no dependent size
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds)to, 16, offset, 0, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (Lds)to, 4, offset, 0, 0, 0);
}
// Waits for all of this wave's loads but the last N.
template <int N>
__device__ inline void loads_done() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// Tokens laid out for the products, in the workspace: 16-byte units, ordered,
// in pieces of 1 KiB, one load of a wave each, which lane takes which unit as
// the instructions want it:
//   few tokens, 16 x 16:  [16 tokens][kt][PIECES p][64 lanes]: lane 16 c + r
//                         takes unit 4 p + c of token r;
//   many, 32 x 32:        [32 tokens][kt][2 PIECES: 2 p + s][64 lanes]: lane
//                         32 h + r takes unit 4 p + 2 h + s of token r.
// For 16 bits also -1.5 2^-8 times each group's sum of each token, [64 tokens]
// [kt][groups][64].  Tokens past m and columns past k are zeros.
constexpr int LAID_TOKENS = 64;   // the workspace holds a multiple of these
__host__ __device__ inline uint64_t laid_units(uint64_t m, uint64_t kt, uint64_t bytes) {
    return (m + LAID_TOKENS - 1) / LAID_TOKENS * LAID_TOKENS * kt * (8 * bytes);
}
inline uint64_t laid_bytes(uint64_t m, uint64_t kt) {   // of the widest type, with sums of the smallest groups
    return laid_units(m, kt, 2) * 16 + (m + LAID_TOKENS - 1) / LAID_TOKENS * LAID_TOKENS * kt * (4 * 4);
}
inline __device__ const u32x4* laid_tokens(const MatvecArgs& a) { return reinterpret_cast<const u32x4*>(a.ws); }
template <typename X>
__device__ inline float* laid_sums(const MatvecArgs& a) {
    return reinterpret_cast<float*>(reinterpret_cast<u32x4*>(a.ws) + laid_units(a.m, a.kt, sizeof(X)));
}

int launch_lay_tokens(const MatvecArgs& a, int x_type, uint32_t group, bool many, hipStream_t s);
constexpr uint32_t MM_TILES = 1u << 22;   // more tiles of columns than this: in the form for few tokens
uint64_t matmul_w4_turns(const MatvecArgs& a);   // its time, in 64 x 64 outputs of a wave
int launch_matmul_w4(const MatvecArgs& a, int x_type, int scale_type, uint32_t group, hipStream_t s);

}  // namespace lecb
