// Declarations shared by the operators of quantised layers: element types,
// conversions on the device, the tile geometry of 4-bit weights, launches.
#pragma once

#include <cstddef>
#include <cstdint>

#include "lecb.h"

namespace lecb {

// 4-bit weights stand in tiles of TILE_ROWS x TILE_COLS codes (lecb.h gives
// the order within a tile): 1 KiB, one 16-byte load of a wave.
constexpr int TILE_ROWS = 16;
constexpr int TILE_COLS = 128;
constexpr int TILE_BYTES = TILE_ROWS * TILE_COLS / 2;

inline uint64_t tiles_of(uint64_t n, uint64_t step) { return n / step + (n % step != 0); }
inline bool valid_group(uint32_t g) { return g == 32 || g == 64 || g == 128; }
inline uint64_t elem_bytes(int type) { return type == LECB_F32 ? 4 : type == LECB_I8 ? 1 : 2; }
inline bool float_type(int t) { return t == LECB_F32 || t == LECB_BF16 || t == LECB_F16; }
inline bool scale_type_ok(int t) { return t == LECB_F32 || t == LECB_BF16; }

struct QuantizeW4 {
    const void* w;
    int type;
    uint64_t stride;
    uint64_t n, k;
    uint32_t group;
    uint8_t* tiles;
    void* scales;
    int scale_type;
};
int launch_quantize_w4(const QuantizeW4& a, void* stream);

struct DequantizeW4 {
    const uint8_t* tiles;
    const void* scales;
    int scale_type;
    uint32_t group;
    uint64_t n, k;
    void* out;
    int type;
    uint64_t stride;
};
int launch_dequantize_w4(const DequantizeW4& a, void* stream);

int launch_tile_w4(const uint8_t* rows, uint8_t* tiles, uint64_t n, uint64_t k, void* stream);
int launch_untile_w4(const uint8_t* tiles, uint8_t* rows, uint64_t n, uint64_t k, void* stream);

struct RmsnormQ8 {
    const void* x;
    uint64_t x_stride;
    const void* res;
    uint64_t res_stride;
    const void* weight;
    int weight_type;
    int type;
    uint64_t rows;
    uint32_t cols;
    float eps;
    void* h;
    uint64_t h_stride;
    int8_t* q;
    float* scale;
    int static_scale;
};
int launch_rmsnorm_q8(const RmsnormQ8& a, void* stream);

int launch_dequantize_q8(const int8_t* q, uint64_t rows, uint64_t cols, const float* scale, int scale_stride,
                         void* out, int type, void* stream);

struct MatvecW4 {
    const void* x;
    int x_type;
    uint64_t x_stride;
    const float* xscale;
    int xscale_stride;
    uint64_t m;
    const uint8_t* tiles;
    const void* scales;
    int scale_type;
    uint32_t group;
    uint64_t n, k;
    void* y;
    int y_type;
    uint64_t y_stride;
    void* ws;
};
int device_cu_count();   // lecb_internal.hpp
uint64_t matvec_w4_workspace(uint64_t m, uint64_t n, uint64_t k);
int launch_matvec_w4(const MatvecW4& a, void* stream);

}  // namespace lecb

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>

namespace lecb {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32_loose __attribute__((aligned(1)));
typedef u32x2 u32x2_loose __attribute__((aligned(1)));
typedef u32x4 u32x4_loose __attribute__((aligned(1)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Eight neighbouring elements as floats, in one 16-byte load or store (two for
// float).  The memory system takes them at any element's address; only the
// last, partial piece of a row goes by elements.
template <typename T>
struct Piece {
    typedef T raw __attribute__((ext_vector_type(16 / sizeof(T))));
    typedef raw loose __attribute__((aligned(sizeof(T))));
    static constexpr int N = sizeof(T) == 4 ? 2 : 1;   // loads
    static constexpr int PER = 8 / N;
    raw v[N];
    __device__ void load(const T* p) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = *reinterpret_cast<const loose*>(p + j * PER);
    }
    // zeros past `count`; entries past it repeat the last one's load (p[0] where
    // there is none: it has to be readable), so that all are in flight at once
    __device__ void load(const T* p, uint64_t count) {
        if (count >= 8) {
            load(p);
        } else {
            T e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = p[(uint64_t)i < count ? i : count ? count - 1 : 0];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i / PER][i % PER] = (uint64_t)i < count ? e[i] : (T)0.0f;
        }
    }
    __device__ float operator[](int i) const { return (float)v[i / PER][i % PER]; }
    __device__ void set(int i, float f) { v[i / PER][i % PER] = (T)f; }   // to nearest, ties to even
    __device__ void store(T* p) const {
#pragma unroll
        for (int j = 0; j < N; ++j) *reinterpret_cast<loose*>(p + j * PER) = v[j];
    }
    __device__ void store(T* p, uint64_t count) const {
        if (count >= 8) {
            store(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((uint64_t)i < count) p[i] = v[i / PER][i % PER];
        }
    }
};

// Calls f with a value of the element type that `type` names (F32, BF16, F16).
template <typename F>
inline int with_float_type(int type, F f) {
    switch (type) {
        case LECB_F32: return f(float());
        case LECB_BF16: return f(__bf16());
        case LECB_F16: return f(_Float16());
        default: return LECB_ERR_INVALID_ARG;
    }
}

inline int launched() { return hipGetLastError() == hipSuccess ? LECB_OK : LECB_ERR_HIP; }

}  // namespace lecb
#endif
