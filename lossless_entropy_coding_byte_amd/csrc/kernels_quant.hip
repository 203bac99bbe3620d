// Rounding to 4 and 8 bits: quantize_w4 / dequantize_w4 / tile_w4 (weights in
// tiles of 4-bit codes), rmsnorm_q8 / dequantize_q8 (activations in int8).
// All of them move their data once and are bound by HBM; lecb.h states the
// formulas and layouts.
#include "layers.hpp"

namespace lecb {

namespace {

constexpr uint32_t ABS_MASK = 0x7fffffffu;
constexpr uint32_t INF_BITS = 0x7f800000u;

// |v| as an unsigned number: orders like |v|, and any NaN above infinity, so
// one unsigned maximum finds both the largest magnitude and what is not finite.
__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & ABS_MASK; }
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// a * b rounded to 32 bits whatever is done with it next: the compiler would
// fuse a product with its conversion to fp16, which rounds once where bf16 and
// the formulas in lecb.h round twice.
__device__ inline float product(float a, float b) {
    float p = a * b;
    asm("" : "+v"(p));
    return p;
}

// ---------------------------------------------------------------- 4-bit weights

// The step of a group and what turns weights into codes.  q = rint(w / s) of
// the exact quotient: with inv = 1 / s rounded, n = rint(w inv) is that or its
// neighbour (w inv is off by under two units in its last place), and e = w - n s
// is exact (one fused operation, and both terms are multiples of the smaller
// one's last place within 24 bits of s), so comparing |e| with s / 2 settles
// it.  Eight weights at a time: what has to be settled is seen from the largest
// |e| of the eight and is rare.  Not so for 16-bit weights with 16-bit steps,
// one in some 700 of which lies half a step between two codes: those settle each
// weight, by adding e / s to n in one more fused operation, with 1/s a little
// smaller where n is even and larger where it is odd, so that half a step goes
// to the even code; any other e differs from it by 2^-12 at least.
//
// Adding MAGIC to w inv, in one fused operation, rounds it to n and leaves n + 8
// in the lowest four bits; shifted and added up, the eight make the word.
// Steps that are not from 2^-60 to 2^100 go one by one, with s and w times 2^64
// where they are small, so that neither 1/s nor s / 2 leaves the range.
struct Step {
    float s;     // as stored (0: all codes 0; NaN: not finite)
    float inv;   // 1 / s, of 2^64 s where s is small, 0 where it is 0 or NaN
    __device__ static float lift(float s) { return s < 0x1p-60f ? 0x1p64f : 1.0f; }
    __device__ void set(uint32_t amax_bits, bool bf16) {
        s = amax_bits >= INF_BITS ? __uint_as_float(0x7fc00000u) : __uint_as_float(amax_bits) / 7.0f;
        if (bf16) s = (float)(__bf16)s;
        // a step that rounding to 16 bits carried to infinity is none either
        if (abs_bits(s) >= INF_BITS) s = __uint_as_float(0x7fc00000u);
        inv = s > 0.0f ? 1.0f / (s * lift(s)) : 0.0f;
    }
    __device__ uint32_t code(float w) const {
        const float t = s * lift(s), v = w * lift(s);
        float n = rintf(v * inv);
        const float e = fmaf(-n, t, v), a = fabsf(e) + fabsf(e);
        const bool odd = ((int)n & 1) != 0;
        if (a > t || (a == t && odd)) n += e > 0.0f ? 1.0f : -1.0f;
        n = fminf(fmaxf(n, -7.0f), 7.0f);
        return inv > 0.0f ? (uint32_t)(int)n & 15u : 0u;
    }
    template <typename P>
    __device__ uint32_t word(const P& w, bool halves) const {   // halves: weights and step of 16 bits
        constexpr float MAGIC = 12582920.0f;   // 1.5 2^23 + 8: 0x4b400008
        uint32_t q = 0u - 0x4b400000u * 0x11111111u;
        float worst = 0.0f;
        if (halves) {
            const uint32_t below = __float_as_uint(inv) - 4;   // units in the last place
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = fmaf(w[i], inv, MAGIC);
                const float e = fmaf(MAGIC - m, s, w[i]);
                m = fmaf(e, __uint_as_float(below + ((__float_as_uint(m) & 1u) << 3)), m);
                q += __float_as_uint(m) << (4 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float m = fmaf(w[i], inv, MAGIC);
                q += __float_as_uint(m) << (4 * i);
                worst = fmaxf(worst, fabsf(fmaf(MAGIC - m, s, w[i])));
            }
        }
        q ^= 0x88888888u;
        if (s == 0.0f) {   // padding, for the most part
            q = 0;
        } else if (!(worst + worst < s && s >= 0x1p-60f && s < 0x1p100f)) {
            q = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) q |= code(w[i]) << (4 * i);
        }
        return q;
    }
};

template <int CTRL>
__device__ inline uint32_t max_lanes(uint32_t v) {   // of v and the v of the lane that CTRL names
    return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}

template <int I>
__device__ inline float of_quad(float v) {   // lane I's of each four
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), I * 0x55, 0xf, 0xf, true));
}

// One wave makes one tile: four loads of four rows each, eight columns a lane,
// so that rows are read in whole lines and a group's maximum is that of 4 to 16
// neighbouring lanes.  Lane i of each four makes the step of load i's row, as the
// two divisions cost as much as four weights' codes.  The words go through LDS
// into the tile's order, so that it leaves in one store.
//
// Bound by HBM, with the vector instructions (about 9 a weight) close behind:
// 8192 x 8192 bf16, groups of 128, 37 us, 4.6 TB/s; fp32, groups of 64, 59 us,
// 5.2 TB/s (a large copy: 5.0).  By 64-byte pieces of 16 rows, as the tile lies,
// the loads and fourteen instructions a weight took 46 and 72 us.
template <typename T, int GROUP>
__global__ __launch_bounds__(256) void quantize_w4_kernel(const T* __restrict__ w, uint64_t stride, uint64_t n,
                                                          uint64_t k, uint32_t kt, uint32_t tiles,
                                                          u32x4* __restrict__ out, void* __restrict__ scales,
                                                          int bf16) {
    constexpr int GROUPS = 128 / GROUP, LANES = GROUP / 8;
    __shared__ __attribute__((aligned(16))) uint32_t s_words[4][4 * 80];   // [c][16 r][4 d], 16 words apart: other banks
    __shared__ float s_scales[4][GROUPS * 16];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile = blockIdx.x * 4 + wave;
    if (tile >= tiles) return;
    const uint32_t lane = threadIdx.x & 63, u = lane & 15;
    const uint32_t tn = tile / kt, tk = tile % kt;
    const uint64_t col = (uint64_t)tk * TILE_COLS + 8 * u;
    const uint64_t left = col < k ? k - col : 0;   // columns from `col` on
    Piece<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t row = (uint64_t)tn * TILE_ROWS + 4 * i + (lane >> 4);
        const uint64_t have = row < n ? left : 0;
        v[i].load(w + (have ? row * stride + col : 0), have);
    }
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) a = umax(a, abs_bits(v[i][e]));
        a = max_lanes<0xB1>(a);                      // the next lane's
        a = max_lanes<0x4E>(a);                      // the next two's
        if (GROUP >= 64) a = max_lanes<0x141>(a);    // mirrored within eight
        if (GROUP >= 128) a = max_lanes<0x140>(a);   // mirrored within sixteen
        mine = (u & 3) == (uint32_t)i ? a : mine;
    }
    Step own;
    own.set(mine, bf16);
    const Step st[4] = {{of_quad<0>(own.s), of_quad<0>(own.inv)}, {of_quad<1>(own.s), of_quad<1>(own.inv)},
                        {of_quad<2>(own.s), of_quad<2>(own.inv)}, {of_quad<3>(own.s), of_quad<3>(own.inv)}};
#pragma unroll
    for (int i = 0; i < 4; ++i) s_words[wave][(u & 3) * 80 + (4 * i + (lane >> 4)) * 4 + (u >> 2)] =
        st[i].word(v[i], sizeof(T) == 2 && bf16);
    if (u % LANES < 4) s_scales[wave][u / LANES * 16 + 4 * (u & 3) + (lane >> 4)] = own.s;
    // one wave's own LDS: its writes come before its reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    out[(uint64_t)tile * 64 + lane] = *reinterpret_cast<const u32x4*>(&s_words[wave][(lane >> 4) * 80 + u * 4]);
    if (lane < GROUPS * 16) {
        const uint64_t at = (uint64_t)tile * (GROUPS * 16) + lane;
        const float s = s_scales[wave][lane];
        if (bf16)
            reinterpret_cast<__bf16*>(scales)[at] = (__bf16)s;
        else
            reinterpret_cast<float*>(scales)[at] = s;
    }
}

__device__ inline float code_value(uint32_t word, int i) { return (float)((int)(word << (28 - 4 * i)) >> 28); }

// A wave a tile; its words go through LDS to lanes that write four whole rows'
// columns at a time, as in quantize_w4_kernel.  Bound by the writes: 8192 x 8192 to
// bf16 in 27 us, 6.2 TB/s with the codes (30 by 64-byte pieces of 16 rows).
template <typename T, int GROUP>
__global__ __launch_bounds__(256) void dequantize_w4_kernel(const u32x4* __restrict__ in,
                                                            const void* __restrict__ scales, int bf16, uint64_t n,
                                                            uint64_t k, uint32_t kt, uint32_t tiles,
                                                            T* __restrict__ out, uint64_t stride) {
    constexpr int GROUPS = 128 / GROUP, LANES = GROUP / 8;
    __shared__ __attribute__((aligned(16))) uint32_t s_words[4][4 * 80];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tile = blockIdx.x * 4 + wave;
    if (tile >= tiles) return;
    const uint32_t lane = threadIdx.x & 63, u = lane & 15;
    *reinterpret_cast<u32x4*>(&s_words[wave][(lane >> 4) * 80 + u * 4]) = in[(uint64_t)tile * 64 + lane];
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t at = ((uint64_t)tile * GROUPS + u / LANES) * 16 + 4 * i + (lane >> 4);
        s[i] = bf16 ? (float)reinterpret_cast<const __bf16*>(scales)[at] : reinterpret_cast<const float*>(scales)[at];
    }
    // one wave's own LDS: its write comes before its reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    const uint64_t col = (uint64_t)(tile % kt) * TILE_COLS + 8 * u;
    if (col >= k) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = 4 * i + (lane >> 4);
        const uint64_t row = (uint64_t)(tile / kt) * TILE_ROWS + r;
        const uint32_t word = s_words[wave][(u & 3) * 80 + r * 4 + (u >> 2)];
        Piece<T> v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, product(code_value(word, e), s[i]));
        if (row < n) v.store(out + row * stride + col, k - col);
    }
}

// Row-major codes <-> tiles: both hold the same 32-bit words, in another order.
// A row's last word may be partial: it goes by bytes, without the unused half.
__global__ __launch_bounds__(256) void tile_w4_kernel(const uint8_t* __restrict__ rows, u32x4* __restrict__ out,
                                                      uint64_t n, uint64_t k, uint32_t kt, uint32_t tiles) {
    const uint32_t tile = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (tile >= tiles) return;
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint64_t row = (uint64_t)(tile / kt) * TILE_ROWS + r;
    const uint64_t col = (uint64_t)(tile % kt) * TILE_COLS + 8 * c;
    const uint64_t pitch = (k + 1) / 2;
    u32x4 words = {0, 0, 0, 0};
    if (row < n) {
        const uint8_t* p = rows + row * pitch;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint64_t c0 = col + 32 * d;
            if (c0 + 8 <= k) {
                words[d] = *reinterpret_cast<const u32_loose*>(p + c0 / 2);
            } else {
                for (uint32_t i = 0; i < 8 && c0 + i < k; ++i)
                    words[d] |= ((uint32_t)p[(c0 + i) / 2] >> (4 * (i & 1)) & 15u) << (4 * i);
            }
        }
    }
    out[(uint64_t)tile * 64 + lane] = words;
}

__global__ __launch_bounds__(256) void untile_w4_kernel(const u32x4* __restrict__ in, uint8_t* __restrict__ rows,
                                                        uint64_t n, uint64_t k, uint32_t kt, uint32_t tiles) {
    const uint32_t tile = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (tile >= tiles) return;
    const uint32_t lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
    const uint64_t row = (uint64_t)(tile / kt) * TILE_ROWS + r;
    const uint64_t col = (uint64_t)(tile % kt) * TILE_COLS + 8 * c;
    const uint64_t pitch = (k + 1) / 2;
    if (row >= n) return;
    const u32x4 words = in[(uint64_t)tile * 64 + lane];
    uint8_t* p = rows + row * pitch;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint64_t c0 = col + 32 * d;
        if (c0 + 8 <= k) {
            *reinterpret_cast<u32_loose*>(p + c0 / 2) = words[d];
        } else {
            for (uint32_t i = 0; i < 8 && c0 + i < k; i += 2) {
                const uint32_t v = words[d] >> (4 * i) & 255u;
                p[(c0 + i) / 2] = (uint8_t)(c0 + i + 1 < k ? v : v & 15u);
            }
        }
    }
}

// ---------------------------------------------------------------- 8-bit activations

// One workgroup of THREADS lanes per row, the row in registers (NV pieces of
// eight elements a lane).  With a = max|h weight|, the scale is a r / 127 for
// r = 1 / sqrt(mean(h^2) + eps) and the codes are rint(h weight 127 / a): r
// cancels, so the sum of squares and the maximum come out of one pass and one
// reduction.  The order of the sums depends on the number of columns alone.
//
// Bound by HBM: 16384 x 2048 bf16 with the residual 40 us, 5.8 TB/s of what it
// reads and writes; 4096 x 8192 fp32 86 us, 5.0 TB/s; one row of 4096 takes
// 3.4 us, two memory latencies and the reduction.
template <int THREADS>
struct RowSums {
    float ss;
    uint32_t amax;
    __device__ void reduce() {
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            ss += __shfl_xor(ss, o);
            amax = umax(amax, __shfl_xor(amax, o));
        }
        if (THREADS > 64) {
            constexpr int W = THREADS / 64;
            __shared__ float s_ss[W];
            __shared__ uint32_t s_max[W];
            __syncthreads();
            if ((threadIdx.x & 63) == 0) {
                s_ss[threadIdx.x >> 6] = ss;
                s_max[threadIdx.x >> 6] = amax;
            }
            __syncthreads();
            ss = s_ss[0];
            amax = s_max[0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                ss += s_ss[i];
                amax = umax(amax, s_max[i]);
            }
        }
    }
};

struct NormArgs {
    const void* x;
    const void* res;
    const void* weight;
    void* h;
    int8_t* q;
    float* scale;
    uint64_t x_stride, res_stride, h_stride;
    uint32_t rows, cols;
    float eps;
    int static_scale;
};

template <typename T, typename W, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void rmsnorm_q8_kernel(NormArgs a) {
    const uint64_t row = blockIdx.x;
    const uint32_t cols = a.cols, c0 = threadIdx.x * 8;
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + row * a.res_stride : nullptr;
    T* h = a.h ? reinterpret_cast<T*>(a.h) + row * a.h_stride : nullptr;
    const W* weight = reinterpret_cast<const W*>(a.weight);
    int8_t* q = a.q + row * cols;
    // everything is asked for before anything is used: a row is as long as one
    // lane's loads take, and h may be where x or the residual is
    float v[NV][8];
    Piece<T> bx[NV], br[NV];
    Piece<W> bw[NV];
#pragma unroll
    for (int p = 0; p < NV; ++p) {
        const uint32_t c = c0 + p * THREADS * 8;
        if (c < cols) {
            bx[p].load(x + c, cols - c);
            if (res) br[p].load(res + c, cols - c);
            bw[p].load(weight + c, cols - c);
        }
    }
    RowSums<THREADS> sums{0.0f, 0u};
#pragma unroll
    for (int p = 0; p < NV; ++p) {
        const uint32_t c = c0 + p * THREADS * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
        if (c < cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[p][i] = bx[p][i];
            if (res) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[p][i] += br[p][i];
            }
            if (h) {
                Piece<T> b;
#pragma unroll
                for (int i = 0; i < 8; ++i) b.set(i, v[p][i]);
                b.store(h + c, cols - c);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sums.ss = fmaf(v[p][i], v[p][i], sums.ss);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[p][i] *= bw[p][i];   // from here on v = h weight
                sums.amax = umax(sums.amax, abs_bits(v[p][i]));
            }
        }
    }
    sums.reduce();
    const float r = 1.0f / sqrtf(sums.ss / (float)cols + a.eps);
    float mul;           // codes are rint(v * lift * mul)
    float lift = 1.0f;
    bool none = false;   // no code but 0
    if (a.static_scale) {
        const float s = a.scale[0];
        none = !(s > 0.0f);
        mul = r / s;
    } else {
        const float amax = __uint_as_float(sums.amax);
        const bool bad = sums.amax >= INF_BITS || abs_bits(sums.ss) >= INF_BITS;
        const float s = bad ? __uint_as_float(0x7fc00000u) : amax * r / 127.0f;
        none = bad || !(s > 0.0f);
        if (amax < 0x1p-60f) lift = 0x1p64f;   // 127 / amax stays in range
        mul = 127.0f / (amax * lift);
        if (threadIdx.x == 0) a.scale[row] = s;
    }
#pragma unroll
    for (int p = 0; p < NV; ++p) {
        const uint32_t c = c0 + p * THREADS * 8;
        if (c >= cols) continue;
        u32x2 b = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = v[p][i] * lift * mul;
            const int code = none || !(y == y) ? 0 : (int)rintf(fminf(fmaxf(y, -127.0f), 127.0f));
            b[i / 4] |= ((uint32_t)code & 255u) << (8 * (i % 4));
        }
        if (cols - c >= 8) {
            *reinterpret_cast<u32x2_loose*>(q + c) = b;
        } else {
            for (uint32_t i = 0; i < cols - c; ++i) q[c + i] = (int8_t)(b[i / 4] >> (8 * (i % 4)));
        }
    }
}

// A lane turns 16 neighbouring codes into values.  They may span rows: two at
// most, whose scales are asked for at once, where rows have 16 columns or more.
// Bound by HBM: 16384 x 2048 to bf16 in 19 us, 5.3 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void dequantize_q8_kernel(const int8_t* __restrict__ q, uint64_t total,
                                                            uint32_t cols, const float* __restrict__ scale,
                                                            int scale_stride, T* __restrict__ out) {
    const uint64_t at = ((uint64_t)blockIdx.x * 256 + threadIdx.x) * 16;
    if (at >= total) return;
    uint64_t row = 0;
    uint32_t left = 16;   // codes of this row
    float s[2] = {scale[0], 0.0f};
    if (scale_stride) {
        // a quotient of 64 bits takes several times as long as one of 32
        row = total <= 0xffffffffu ? (uint32_t)at / cols : at / cols;
        left = (uint32_t)((row + 1) * cols - at);
        s[0] = scale[row];
        s[1] = scale[row + (at + left < total)];
    }
    const bool whole = at + 16 <= total;
    u32x4 b = {0, 0, 0, 0};
    if (whole) {
        b = *reinterpret_cast<const u32x4*>(q + at);
    } else {
        for (uint32_t i = 0; at + i < total; ++i) b[i / 4] |= (uint32_t)(uint8_t)q[at + i] << (8 * (i % 4));
    }
    Piece<T> v[2];
    if (cols >= 16 || !scale_stride) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i / 8].set(i % 8, product((float)((int)(b[i / 4] << (24 - 8 * (i % 4))) >> 24), (uint32_t)i < left ? s[0] : s[1]));
    } else {
        float f = s[0];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i / 8].set(i % 8, product((float)((int)(b[i / 4] << (24 - 8 * (i % 4))) >> 24), f));
            if (--left == 0 && at + i + 1 < total) {
                left = cols;
                f = scale[++row];
            }
        }
    }
    v[0].store(out + at, total - at);
    if (total - at > 8) v[1].store(out + at + 8, total - at - 8);
}

// A launch has fewer than 2^32 lanes: more rows than that go by several.
template <typename T, typename W, int THREADS, int NV>
int launch_norm_rows(NormArgs a, hipStream_t s) {
    constexpr uint32_t MOST = (1u << 31) / THREADS;
    for (uint32_t left = a.rows; left;) {
        const uint32_t rows = left < MOST ? left : MOST;
        rmsnorm_q8_kernel<T, W, THREADS, NV><<<dim3(rows), THREADS, 0, s>>>(a);
        const int rc = launched();
        if (rc) return rc;
        left -= rows;
        a.x = static_cast<const T*>(a.x) + rows * a.x_stride;
        if (a.res) a.res = static_cast<const T*>(a.res) + rows * a.res_stride;
        if (a.h) a.h = static_cast<T*>(a.h) + rows * a.h_stride;
        a.q += (uint64_t)rows * a.cols;
        if (!a.static_scale) a.scale += rows;
    }
    return LECB_OK;
}

template <typename T, typename W>
int launch_norm_as(const NormArgs& a, hipStream_t s) {
    const uint32_t pieces = (a.cols + 7) / 8;
    if (pieces <= 64) return launch_norm_rows<T, W, 64, 1>(a, s);
    if (pieces <= 256) return launch_norm_rows<T, W, 256, 1>(a, s);
    if (pieces <= 1024) return launch_norm_rows<T, W, 256, 4>(a, s);
    return launch_norm_rows<T, W, 1024, 4>(a, s);
}

// Rows of 4-bit weights that one launch takes, a wave a tile: it has fewer than
// 2^32 lanes.
struct Share {
    uint64_t row, rows, first_tile;
    uint32_t kt, tiles;
    dim3 grid() const { return dim3((tiles + 3) / 4); }
};
template <typename F>
int by_rows(uint64_t n, uint64_t k, F launch) {
    const uint64_t kt = tiles_of(k, TILE_COLS), most = (1ull << 25) / kt * TILE_ROWS;   // kt: 2^24 at most
    for (uint64_t row = 0; row < n; row += most) {
        const uint64_t rows = n - row < most ? n - row : most;
        launch(Share{row, rows, row / TILE_ROWS * kt, (uint32_t)kt, (uint32_t)(tiles_of(rows, TILE_ROWS) * kt)});
        const int rc = launched();
        if (rc) return rc;
    }
    return LECB_OK;
}

}  // namespace

int launch_quantize_w4(const QuantizeW4& a, void* stream) {
    return with_float_type(a.type, [&](auto t) -> int {
        typedef decltype(t) T;
        auto go = [&](auto group) {
            constexpr int G = decltype(group)::value;
            return by_rows(a.n, a.k, [&](const Share& p) {
                const uint64_t at = p.first_tile * (128 / G * TILE_ROWS) * (a.scale_type == LECB_BF16 ? 2 : 4);
                quantize_w4_kernel<T, G><<<p.grid(), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
                    static_cast<const T*>(a.w) + p.row * a.stride, a.stride, p.rows, a.k, p.kt, p.tiles,
                    reinterpret_cast<u32x4*>(a.tiles) + p.first_tile * 64, static_cast<char*>(a.scales) + at,
                    a.scale_type == LECB_BF16);
            });
        };
        if (a.group == 32) return go(std::integral_constant<int, 32>());
        if (a.group == 64) return go(std::integral_constant<int, 64>());
        return go(std::integral_constant<int, 128>());
    });
}

int launch_dequantize_w4(const DequantizeW4& a, void* stream) {
    return with_float_type(a.type, [&](auto t) -> int {
        typedef decltype(t) T;
        auto go = [&](auto group) {
            constexpr int G = decltype(group)::value;
            return by_rows(a.n, a.k, [&](const Share& p) {
                const uint64_t at = p.first_tile * (128 / G * TILE_ROWS) * (a.scale_type == LECB_BF16 ? 2 : 4);
                dequantize_w4_kernel<T, G><<<p.grid(), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
                    reinterpret_cast<const u32x4*>(a.tiles) + p.first_tile * 64,
                    static_cast<const char*>(a.scales) + at, a.scale_type == LECB_BF16, p.rows, a.k, p.kt, p.tiles,
                    static_cast<T*>(a.out) + p.row * a.stride, a.stride);
            });
        };
        if (a.group == 32) return go(std::integral_constant<int, 32>());
        if (a.group == 64) return go(std::integral_constant<int, 64>());
        return go(std::integral_constant<int, 128>());
    });
}

int launch_tile_w4(const uint8_t* rows, uint8_t* tiles, uint64_t n, uint64_t k, void* stream) {
    return by_rows(n, k, [&](const Share& p) {
        tile_w4_kernel<<<p.grid(), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
            rows + p.row * ((k + 1) / 2), reinterpret_cast<u32x4*>(tiles) + p.first_tile * 64, p.rows, k, p.kt, p.tiles);
    });
}

int launch_untile_w4(const uint8_t* tiles, uint8_t* rows, uint64_t n, uint64_t k, void* stream) {
    return by_rows(n, k, [&](const Share& p) {
        untile_w4_kernel<<<p.grid(), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
            reinterpret_cast<const u32x4*>(tiles) + p.first_tile * 64, rows + p.row * ((k + 1) / 2), p.rows, k, p.kt,
            p.tiles);
    });
}

int launch_rmsnorm_q8(const RmsnormQ8& a, void* stream) {
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const NormArgs b = {a.x, a.res, a.weight, a.h, a.q, a.scale, a.x_stride, a.res_stride, a.h_stride,
                        (uint32_t)a.rows, a.cols, a.eps, a.static_scale};
    return with_float_type(a.type, [&](auto t) -> int {
        return with_float_type(a.weight_type, [&](auto w) -> int {
            return launch_norm_as<decltype(t), decltype(w)>(b, s);
        });
    });
}

int launch_dequantize_q8(const int8_t* q, uint64_t rows, uint64_t cols, const float* scale, int scale_stride,
                         void* out, int type, void* stream) {
    const uint64_t total = rows * cols;
    const dim3 grid((uint32_t)((total + 4095) / 4096));
    return with_float_type(type, [&](auto t) -> int {
        typedef decltype(t) T;
        dequantize_q8_kernel<T><<<grid, 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(
            q, total, (uint32_t)cols, scale, scale_stride, static_cast<T*>(out));
        return launched();
    });
}

}  // namespace lecb
