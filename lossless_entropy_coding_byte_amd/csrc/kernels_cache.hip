// The 8-bit cache of keys and values: new tokens into its blocks
// (cache_write_q8) and rows back out of them (cache_read_q8).  lecb.h states
// layouts and formulas.
#include "cache.hpp"

namespace lecb {

namespace {

constexpr uint32_t ABS_MASK = 0x7fffffffu;
constexpr uint32_t INF_BITS = 0x7f800000u;
constexpr int THREADS = 256;

__device__ inline uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// a * b rounded to 32 bits before anything else is done with it.
__device__ inline float product(float a, float b) {
    float p = a * b;
    asm("" : "+v"(p));
    return p;
}

// What a workgroup works on: rows of one sequence within one block.
//
// Workgroup w of `items` finds its sequence without a sum over the others: the rows of
// sequence s touch at most (rows - 1) / block + 2 blocks, so it owns the numbers
// from starts[s] / block + 2 s on, up to those of sequence s + 1.
struct Span {
    uint32_t seq, index, page;   // sequence, its block, the cache's
    uint32_t lo, hi;             // tokens lo .. hi - 1 of the block are rows; none: lo == hi
    uint32_t row;                // of token lo
    bool bad;
    __device__ bool find(const Seqs& q, uint32_t w) {
        uint32_t s = 0, skip = 0;
        if (q.starts) {
            uint32_t end = q.seqs;   // the last sequence whose numbers begin at w or before
            while (end - s > 1) {
                const uint32_t mid = (s + end) / 2;
                if (q.begin(mid) / q.block + 2 * mid <= w)
                    s = mid;
                else
                    end = mid;
            }
            skip = w - (q.begin(s) / q.block + 2 * s);   // starts that do not rise wrap around: past every block
        } else {
            s = w;
        }
        const uint32_t n = q.count(s), len = q.length(s);
        seq = s;
        bad = q.bad(len);
        const uint32_t first = len > n ? len - n : 0;   // tokens first .. len - 1
        const uint64_t j = (uint64_t)first / q.block + skip;
        if (j * q.block >= len || n == 0) return false;
        index = (uint32_t)j;
        const uint32_t at = index * q.block;
        lo = first > at ? first - at : 0;
        hi = umin(len - at, q.block);
        row = q.begin(s) + (at + lo - len + n);   // n > len: the first rows have no token
        page = bad ? 0xffffffffu : q.page(s, index);
        bad = bad || page >= q.blocks;
        return true;
    }
};

// Byte of a unit that holds token t, dimension d of it.
__device__ inline uint32_t key_byte(uint32_t t, uint32_t d) {
    return ((d / 8 * 16 + t % 16) * 2 + t / 16) * 8 + d % 8;
}
__device__ inline uint32_t value_byte(uint32_t t, uint32_t d) {
    return ((t % 16 / 4 * 16 + d % 16) * 2 + d / 16) * 8 + t / 16 * 4 + t % 4;
}

// A block's scale and what turns numbers into codes: q = rint(x / s) of the
// exact quotient.  With inv = 1 / s rounded, n = rint(x inv) is that or its
// neighbour, e = x - n s is exact in one fused operation, and comparing |e| with
// s / 2 settles it.  Scales below 2^-60 go times 2^64, so that 1 / s stays in range.
struct Step {
    float s, inv, t, lift;
    __device__ void set(float scale) {
        s = scale;
        lift = s < 0x1p-60f ? 0x1p64f : 1.0f;
        t = s * lift;
        inv = s > 0.0f && s < __uint_as_float(INF_BITS) ? 1.0f / t : 0.0f;
    }
    __device__ int code(float x) const {
        const float v = x * lift;
        float n = rintf(v * inv);
        const float e = fmaf(-n, t, v), a = fabsf(e) + fabsf(e);
        if (a > t || (a == t && ((int)n & 1))) n += e > 0.0f ? 1.0f : -1.0f;
        n = fminf(fmaxf(n, -127.0f), 127.0f);
        return inv > 0.0f ? (int)n : 0;
    }
};

struct WriteArgs {
    Seqs seqs;
    const void* x[2];
    uint64_t token[2], head[2];   // strides
    uint8_t* codes[2];
    float* scale[2];
    uint32_t heads, dim, units;
};

// A workgroup writes the rows of one span for one head, keys or values: their
// largest magnitude first, then the codes by tiles of 32 tokens, put together in
// LDS in the order of a tile and stored by 16-byte pieces.
template <typename T>
__global__ __launch_bounds__(THREADS) void cache_write_kernel(WriteArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_tile[8 * UNIT_BYTES];
    __shared__ uint32_t s_max[THREADS / 64];
    Span p;
    if (!p.find(a.seqs, blockIdx.x) || p.bad) return;
    const uint32_t which = blockIdx.z, h = blockIdx.y, block = a.seqs.block;
    const uint64_t cell = (uint64_t)p.page * a.heads + h;
    const T* x = reinterpret_cast<const T*>(a.x[which]) + h * a.head[which];
    const uint64_t stride = a.token[which];
    const uint32_t pieces = (a.dim + 7) / 8, count = (p.hi - p.lo) * pieces;

    uint32_t amax = 0;
    for (uint32_t i = threadIdx.x; i < count; i += THREADS) {
        const uint32_t t = i / pieces, d = i % pieces * 8;
        Piece<T> v;
        v.load(x + (uint64_t)(p.row + t) * stride + d, a.dim - d);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = umax(amax, __float_as_uint(v[e]) & ABS_MASK);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) amax = umax(amax, (uint32_t)__shfl_xor((int)amax, o));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x / 64] = amax;
    const float was = a.scale[which][cell];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) amax = umax(amax, s_max[i]);
    const float need = amax >= INF_BITS ? __uint_as_float(0x7fc00000u) : __uint_as_float(amax) / 127.0f;
    const bool kept = p.lo > 0;
    float scale = need;
    if (kept && need <= was) scale = was;
    if (kept && need > was) scale = fmaxf(need, 1.25f * was);
    if (kept && !(was == was)) scale = was;
    const bool grow = kept && __float_as_uint(scale) != __float_as_uint(was);
    if (threadIdx.x == 0) a.scale[which][cell] = scale;
    Step step;
    step.set(scale);

    const uint32_t tile_bytes = a.units * UNIT_BYTES;
    uint8_t* out = a.codes[which] + cell * (block / TILE_TOKENS) * tile_bytes;
    for (uint32_t tile = grow ? 0 : p.lo / TILE_TOKENS; tile * TILE_TOKENS < p.hi; ++tile) {
        const uint32_t begin = tile * TILE_TOKENS;
        u32x4* mem = reinterpret_cast<u32x4*>(out + (uint64_t)tile * tile_bytes);
        for (uint32_t i = threadIdx.x; i < tile_bytes / 16; i += THREADS) {
            u32x4 w = {0, 0, 0, 0};
            if (begin < p.lo) w = mem[i];
            if (grow) {
                // codes of 8 bits by scales of 24: exact quotients in 64 bits never lie so near to half a step that rounding could cross it
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t r = 0;
#pragma unroll
                    for (int b = 0; b < 32; b += 8) {
                        const double v = (double)(int8_t)(w[j] >> b) * (double)was / (double)scale;
                        const int q = step.inv > 0.0f ? (int)fmin(fmax(rint(v), -127.0), 127.0) : 0;
                        r |= (uint32_t)(q & 255) << b;
                    }
                    w[j] = r;
                }
            }
            reinterpret_cast<u32x4*>(s_tile)[i] = w;
        }
        __syncthreads();
        const uint32_t from = begin > p.lo ? begin : p.lo, to = umin(begin + TILE_TOKENS, p.hi);
        if (from < to) {
            const uint32_t n = (to - from) * pieces;
            for (uint32_t i = threadIdx.x; i < n; i += THREADS) {
                const uint32_t t = from + i / pieces, d = i % pieces * 8;
                Piece<T> v;
                v.load(x + (uint64_t)(p.row + t - p.lo) * stride + d, a.dim - d);
                uint32_t q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = (uint32_t)step.code(v[e]) & 255u;
                uint8_t* unit = s_tile + d / 32 * UNIT_BYTES;
                if (which == 0) {
                    u32x2 w = {q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24};
                    *reinterpret_cast<u32x2*>(unit + key_byte(t % TILE_TOKENS, d % 32)) = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) unit[value_byte(t % TILE_TOKENS, d % 32 + e)] = (uint8_t)q[e];
                }
            }
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < tile_bytes / 16; i += THREADS) mem[i] = reinterpret_cast<u32x4*>(s_tile)[i];
        __syncthreads();
    }
}

struct ReadArgs {
    Seqs seqs;
    const uint8_t* codes[2];
    const float* scale[2];
    void* out[2];
    uint32_t heads, dim, units;
    uint32_t items;   // workgroups past them: rows without a token
    int fill;
};

template <typename T>
__device__ void put_row(T* out, uint32_t dim, float v) {
    for (uint32_t d = threadIdx.x; d < dim; d += THREADS) out[d] = (T)v;
}

template <typename T>
__global__ __launch_bounds__(THREADS) void cache_read_kernel(ReadArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_tile[8 * UNIT_BYTES];
    const uint32_t which = blockIdx.z, h = blockIdx.y, block = a.seqs.block;
    T* out = reinterpret_cast<T*>(a.out[which]) + (uint64_t)h * a.dim;
    const uint64_t stride = (uint64_t)a.heads * a.dim;
    if (blockIdx.x >= a.items) {
        const uint32_t me = blockIdx.x - a.items, all = gridDim.x - a.items;
        uint32_t second = 0;
        const uint32_t b = a.seqs.starts ? a.seqs.begin(0) : 0, n = a.fill ? a.seqs.outside(&second) : 0;
        for (uint32_t i = me; i < n; i += all) put_row(out + (uint64_t)(i < b ? i : second + i - b) * stride, a.dim, 0.0f);
        // rows of a sequence before its first token
        for (uint32_t s = me; s < a.seqs.seqs; s += all) {
            const uint32_t rows = a.seqs.count(s), len = a.seqs.length(s);
            for (uint32_t i = 0; i + len < rows; ++i) put_row(out + (uint64_t)(a.seqs.begin(s) + i) * stride, a.dim, 0.0f);
        }
        return;
    }
    Span p;
    if (!p.find(a.seqs, blockIdx.x)) return;
    if (p.bad) {
        for (uint32_t i = 0; i < p.hi - p.lo; ++i)
            put_row(out + (uint64_t)(p.row + i) * stride, a.dim, __uint_as_float(0x7fc00000u));
        return;
    }
    const uint64_t cell = (uint64_t)p.page * a.heads + h;
    const uint32_t pieces = (a.dim + 7) / 8, tile_bytes = a.units * UNIT_BYTES;
    const uint8_t* in = a.codes[which] + cell * (block / TILE_TOKENS) * tile_bytes;
    const float scale = a.scale[which][cell];
    for (uint32_t tile = p.lo / TILE_TOKENS; tile * TILE_TOKENS < p.hi; ++tile) {
        const uint32_t begin = tile * TILE_TOKENS;
        const u32x4* mem = reinterpret_cast<const u32x4*>(in + (uint64_t)tile * tile_bytes);
        for (uint32_t i = threadIdx.x; i < tile_bytes / 16; i += THREADS) reinterpret_cast<u32x4*>(s_tile)[i] = mem[i];
        __syncthreads();
        const uint32_t from = begin > p.lo ? begin : p.lo, to = umin(begin + TILE_TOKENS, p.hi);
        const uint32_t n = (to - from) * pieces;
        for (uint32_t i = threadIdx.x; i < n; i += THREADS) {
            const uint32_t t = from + i / pieces, d = i % pieces * 8;
            const uint8_t* unit = s_tile + d / 32 * UNIT_BYTES;
            Piece<T> v;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t at = which == 0 ? key_byte(t % TILE_TOKENS, d % 32) + e : value_byte(t % TILE_TOKENS, d % 32 + e);
                v.set(e, product((float)(int8_t)unit[at], scale));
            }
            v.store(out + (uint64_t)(p.row + t - p.lo) * stride + d, a.dim - d);
        }
        __syncthreads();
    }
}

uint64_t items_of(const lecb_cache_q8& c, const lecb_cache_seqs& s) {
    return s.starts ? (uint64_t)s.tokens / c.block + 2ull * s.seqs : s.seqs;
}

}  // namespace

int launch_cache_write_q8(const lecb_cache_q8& c, const lecb_cache_seqs& s, const void* k, const void* v, int type,
                          uint64_t k_token, uint64_t k_head, uint64_t v_token, uint64_t v_head, void* stream) {
    const WriteArgs a = {seqs_of(c, s), {k, v}, {k_token, v_token}, {k_head, v_head},
                         {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v)}, {c.k_scale, c.v_scale},
                         c.heads, c.dim, padded_dim(c.dim) / 32};
    return with_float_type(type, [&](auto t) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(cache_write_kernel<decltype(t)>), dim3((uint32_t)items_of(c, s), c.heads, 2),
                           dim3(THREADS), 0, static_cast<hipStream_t>(stream), a);
        return launched();
    });
}

int launch_cache_read_q8(const lecb_cache_q8& c, const lecb_cache_seqs& s, void* k, void* v, int type, int fill,
                         void* stream) {
    const uint32_t items = (uint32_t)items_of(c, s);
    // without starts a row may still have no token (length 0)
    const uint32_t more = s.starts ? (s.tokens + 15) / 16 < 64 ? (s.tokens + 15) / 16 : 64 : (s.seqs + 63) / 64;
    const ReadArgs a = {seqs_of(c, s), {static_cast<const uint8_t*>(c.k), static_cast<const uint8_t*>(c.v)},
                        {c.k_scale, c.v_scale}, {k, v}, c.heads, c.dim, padded_dim(c.dim) / 32, items, fill};
    return with_float_type(type, [&](auto t) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(cache_read_kernel<decltype(t)>), dim3(items + more, c.heads, 2), dim3(THREADS),
                           0, static_cast<hipStream_t>(stream), a);
        return launched();
    });
}

}  // namespace lecb
