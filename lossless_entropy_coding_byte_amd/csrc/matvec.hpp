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
// columns and the odd ones in a register each.  FACTOR, of the result, undoes 16.
//
// 16 bits: every code as the number it is, for errors that follow the sum of
// |x q|: a column whose code is 0 adds nothing, however large x is there.  A
// code's magnitude (0..8) and sign in a byte are the e4m3 number q 2^-9, as
// that type's numbers are evenly spaced up to 2^-5: nine logic operations and
// additions make the bytes of eight codes, four conversions (scaled, exact) their
// pairs.  (An offset that turns a code's bits into a number's by one operation a
// pair takes eight in all, but has to cancel out of the sums: 24 times the
// tokens', whose rounding is left.)
//
// bf16: q 2^-10 keeps a group's sum (128 x 8) within the range of x; its
// smallest numbers' products, multiples of 2^-143, are still exact.  SCALE, of a
// group's scale, undoes it.  fp16: q, as no sum of it leaves the range.
template <typename X>
struct Operand;

// The bytes described above: of the even columns and of the odd ones.  Three-input
// logic operations take half as long as the and-ors that the compiler makes of this.
__device__ inline u32x2 code_bytes(uint32_t w) {
    constexpr uint32_t PICK = 0xE4, TURN = 0x6C;   // c ? a : b and (a & c) ^ b, bit by bit
    const uint32_t sign = w & 0x88888888u, one = sign >> 3;
    const uint32_t size = __builtin_amdgcn_bitop3_b32(w, sign - one, 0x77777777u, TURN) + one;
    return {(uint32_t)__builtin_amdgcn_bitop3_b32(size, sign << 4, 0x0F0F0F0Fu, PICK),
            (uint32_t)__builtin_amdgcn_bitop3_b32(size >> 4, sign, 0x0F0F0F0Fu, PICK)};
}
// Eight halves in the order of those bytes' pairs: 0 2, 4 6, 1 3, 5 7.
__device__ inline u32x4 pairs_of_halves(u32x4 x) {
    return {__builtin_amdgcn_perm(x.y, x.x, 0x05040100u), __builtin_amdgcn_perm(x.w, x.z, 0x05040100u),
            __builtin_amdgcn_perm(x.y, x.x, 0x07060302u), __builtin_amdgcn_perm(x.w, x.z, 0x07060302u)};
}

template <>
struct Operand<__bf16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float SCALE = 1024.0f, FACTOR = 1.0f;
    static __device__ A weights(uint32_t w) {
        const u32x2 b = code_bytes(w);
        auto pair = [](bf16x2 v) { return __builtin_bit_cast(uint32_t, v); };
        return {pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 0.5f, false)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.x, 0.5f, true)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 0.5f, false)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b.y, 0.5f, true))};
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
};
template <>
struct Operand<_Float16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float SCALE = 1.0f, FACTOR = 1.0f;
    static __device__ A weights(uint32_t w) {
        const u32x2 b = code_bytes(w);
        auto pair = [](f16x2 v) { return __builtin_bit_cast(uint32_t, v); };
        return {pair(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b.x, 512.0f, false)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b.x, 512.0f, true)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b.y, 512.0f, false)),
                pair(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b.y, 512.0f, true))};
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
};
template <>
struct Operand<int8_t> {
    typedef u32x2 A;
    typedef i32x4 Acc;
    static constexpr float SCALE = 1.0f, FACTOR = 0.0625f;
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
// Tokens past m and columns past k are zeros.
constexpr int LAID_TOKENS = 64;   // the workspace holds a multiple of these
__host__ __device__ inline uint64_t laid_units(uint64_t m, uint64_t kt, uint64_t bytes) {
    return (m + LAID_TOKENS - 1) / LAID_TOKENS * LAID_TOKENS * kt * (8 * bytes);
}
inline uint64_t laid_bytes(uint64_t m, uint64_t kt) { return laid_units(m, kt, 2) * 16; }   // of the widest type
inline __device__ const u32x4* laid_tokens(const MatvecArgs& a) { return reinterpret_cast<const u32x4*>(a.ws); }

constexpr uint64_t LAY_ACROSS = 1u << 21;   // workgroups along the columns of one launch
int launch_lay_tokens(const MatvecArgs& a, int x_type, bool many, hipStream_t s);
constexpr uint32_t MM_TILES = 1u << 22;   // more tiles of columns than this: in the form for few tokens
uint64_t matmul_w4_turns(const MatvecArgs& a);   // its time, in 64 x 64 outputs of a wave
int launch_matmul_w4(const MatvecArgs& a, int x_type, int scale_type, uint32_t group, hipStream_t s);

}  // namespace lecb
