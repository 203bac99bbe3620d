// What the products with 4-bit weights share: matrix instructions' operands out
// of codes and tokens, loads of tokens, the last rounding.
#pragma once

#include "layers.hpp"

namespace lecb {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// A word's eight codes as the matrix instruction's operand, eight entries of x
// as the other, and their product.
//
// 16-bit x: the codes become q / 16, exactly: one conversion each (the even
// codes from the word, the odd ones from the word shifted by four, byte by
// byte) and one packing per pair.  int8 x: a code's four bits as the upper
// half of a byte, 16 q, even columns and odd columns in a register each; x is
// put into the same order.  FACTOR takes the sixteen off again, exactly.
template <typename X>
struct Operand;

__device__ inline void code_floats(uint32_t w, float* f) {   // f[i] = code i / 16
    uint32_t u = w >> 4;
    asm("" : "+v"(u));   // keeps one shift, so that every other conversion picks its byte itself
    f[0] = __builtin_amdgcn_cvt_off_f32_i4(w);
    f[1] = __builtin_amdgcn_cvt_off_f32_i4(u);
    f[2] = __builtin_amdgcn_cvt_off_f32_i4((w >> 8) & 255u);
    f[3] = __builtin_amdgcn_cvt_off_f32_i4((u >> 8) & 255u);
    f[4] = __builtin_amdgcn_cvt_off_f32_i4(w >> 16);
    f[5] = __builtin_amdgcn_cvt_off_f32_i4(u >> 16);
    f[6] = __builtin_amdgcn_cvt_off_f32_i4(w >> 24);
    f[7] = __builtin_amdgcn_cvt_off_f32_i4(u >> 24);
}

template <>
struct Operand<__bf16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float FACTOR = 16.0f;
    static __device__ A weights(uint32_t w) {
        float f[8];
        code_floats(w, f);
        A a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
        return a;
    }
    static __device__ A tokens(A x) { return x; }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
};
template <>
struct Operand<_Float16> {
    typedef u32x4 A;
    typedef f32x4 Acc;
    static constexpr float FACTOR = 16.0f;
    static __device__ A weights(uint32_t w) {
        float f[8];
        code_floats(w, f);
        A a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            a[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2 * i], f[2 * i + 1]));
        return a;
    }
    static __device__ A tokens(A x) { return x; }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    }
};
template <>
struct Operand<int8_t> {
    typedef u32x2 A;
    typedef i32x4 Acc;
    static constexpr float FACTOR = 0.0625f;
    static __device__ A weights(uint32_t w) { return {(w << 4) & 0xF0F0F0F0u, w & 0xF0F0F0F0u}; }
    static __device__ A tokens(A x) {
        return {__builtin_amdgcn_perm(x.y, x.x, 0x06040200u), __builtin_amdgcn_perm(x.y, x.x, 0x07050301u)};
    }
    static __device__ Acc mul(A a, A b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0,
                                                     0, 0);
    }
    // two words at once: 64 columns an instruction, at twice the rate
    static __device__ Acc mul2(A a0, A a1, A b0, A b1, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{(int)a0.x, (int)a0.y, (int)a1.x, (int)a1.y},
                                                     i32x4{(int)b0.x, (int)b0.y, (int)b1.x, (int)b1.y}, c, 0, 0, 0);
    }
};

// Eight entries of a row of x; the guarded form takes `count` of them (zeros
// past that) and is used where a row's last tile is partial.
template <typename X>
__device__ inline typename Operand<X>::A load_x8(const X* p) {
    typedef typename Operand<X>::A A;
    typedef A loose __attribute__((aligned(sizeof(X))));
    return *reinterpret_cast<const loose*>(p);
}
template <typename X>
__device__ inline typename Operand<X>::A load_x8(const X* p, uint64_t count) {
    if (count >= 8) return load_x8(p);
    typename Operand<X>::A v{};
    constexpr int PER = 4 / sizeof(X), BITS = 8 * sizeof(X);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if ((uint64_t)i >= count) continue;
        const uint32_t e = sizeof(X) == 1 ? reinterpret_cast<const uint8_t*>(p)[i]
                                          : reinterpret_cast<const uint16_t*>(p)[i];
        v[i / PER] |= e << (BITS * (i % PER));
    }
    return v;
}

// Four neighbouring scales as loaded, and as numbers.
template <typename S>
struct Scales {
    typedef S raw __attribute__((ext_vector_type(4)));
    raw v;
    __device__ void load(const S* p) { v = *reinterpret_cast<const raw*>(p); }
    __device__ float operator[](int i) const { return (float)v[i]; }
};

// The last step of a sum: the token's factor, one rounding, four outputs.
__device__ inline void store_y(void* y, int type, uint64_t at, uint64_t left, f32x4 v) {
    if (left >= 4) {
        if (type == LECB_F32) {
            typedef f32x4 loose __attribute__((aligned(4)));
            *reinterpret_cast<loose*>(reinterpret_cast<float*>(y) + at) = v;
        } else if (type == LECB_BF16) {
            typedef bf16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<__bf16*>(y) + at) =
                bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
            typedef f16x4 loose __attribute__((aligned(2)));
            *reinterpret_cast<loose*>(reinterpret_cast<_Float16*>(y) + at) =
                f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if ((uint64_t)e >= left) continue;
        if (type == LECB_F32)
            reinterpret_cast<float*>(y)[at + e] = v[e];
        else if (type == LECB_BF16)
            reinterpret_cast<__bf16*>(y)[at + e] = (__bf16)v[e];
        else
            reinterpret_cast<_Float16*>(y)[at + e] = (_Float16)v[e];
    }
}

struct MatvecArgs {
    const void* x;
    const float* xscale;
    const u32x4* tiles;
    const void* scales;
    void* y;
    uint64_t x_stride, y_stride, n, k, m;
    uint32_t nt, kt;
    int xscale_stride, y_type;
};

int launch_matmul_w4(const MatvecArgs& a, int x_type, int scale_type, uint32_t group, hipStream_t s);

}  // namespace lecb
