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
    // Called by whole waves: 64 sequences are looked at in one load, so that 4096 take two.
    __device__ bool find(const Seqs& q, uint32_t w, uint32_t lane) {
        uint32_t s = 0, skip = 0, begin, n, len;
        if (q.starts) {
            uint32_t step = 1;
            while ((uint64_t)step * 64 < q.seqs) step *= 64;
            for (;; step /= 64) {   // the last sequence whose numbers begin at w or before
                const uint32_t mine = umin(s + lane * step, q.seqs - 1);
                begin = q.begin(mine);
                n = q.count(mine);   // what the last round needs of the one that it finds
                len = q.length(mine);
                const uint64_t after = __ballot(lane > 0 && (s + lane * step >= q.seqs || begin / q.block + 2 * mine > w));
                const int at = (after ? __builtin_ctzll(after) : 64) - 1;
                s = __builtin_amdgcn_readfirstlane(s + at * step);
                if (step > 1) continue;
                begin = __builtin_amdgcn_readlane(begin, at);
                n = __builtin_amdgcn_readlane(n, at);
                len = __builtin_amdgcn_readlane(len, at);
                break;
            }
            skip = w - (begin / q.block + 2 * s);   // starts that do not rise wrap around: past every block
        } else {
            s = begin = w;
            n = 1;
            len = q.length(s);
        }
        seq = s;
        bad = q.bad(len);
        const uint32_t first = len > n ? len - n : 0;   // tokens first .. len - 1
        const uint64_t j = (uint64_t)first / q.block + skip;
        if (j * q.block >= len || n == 0) return false;
        index = (uint32_t)j;
        const uint32_t at = index * q.block;
        lo = first > at ? first - at : 0;
        hi = umin(len - at, q.block);
        row = begin + (at + lo - len + n);   // n > len: the first rows have no token
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
    float inv, t, lift;   // 1 / t, 0 where there is none; t = s lift
    __device__ void set(float s) {
        lift = s < 0x1p-60f ? 0x1p64f : 1.0f;
        t = s * lift;
        inv = s > 0.0f && s < __uint_as_float(INF_BITS) ? 1.0f / t : 0.0f;
    }
};

// Eight codes, in the order of their bytes.  Adding MAGIC to x inv, in one fused
// operation, rounds it to n and leaves n in the lowest byte.  Where the largest |e|
// of the eight does not settle them (16-bit numbers are half of the block's
// largest, half a step between two codes, often enough), n moves towards e if
// |e| > s / 2, or |e| = s / 2 and n is odd.
__device__ inline u32x2 codes_of(const Step& k, const float (&x)[8]) {
    constexpr float MAGIC = 12582912.0f;   // 1.5 2^23
    if (!(k.inv > 0.0f)) return u32x2{0, 0};
    float worst = 0.0f;
    uint32_t m[8];
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = x[i] * k.lift, f = fmaf(v, k.inv, MAGIC);
        m[i] = __float_as_uint(f);
        e[i] = fmaf(MAGIC - f, k.t, v);
        worst = fmaxf(worst, fabsf(e[i]));
    }
    const float half = 0.5f * k.t;
    if (worst >= half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(e[i]);
            const bool off = (b & ABS_MASK) + (m[i] & 1) > __float_as_uint(half);
            m[i] += off ? (uint32_t)((int)b >> 31 | 1) : 0;
        }
    }
    if (k.lift != 1.0f) {   // a scale rounded down at the bottom of the range leaves more than 127 steps
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = (int)(m[i] - __float_as_uint(MAGIC));
            m[i] = (uint32_t)(n > 127 ? 127 : n < -127 ? -127 : n);
        }
    }
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x0c0c0400u);
        w[i] = lo | hi << 16;
    }
    return w;
}

struct WriteArgs {
    Seqs seqs;
    const void* x[2];
    uint64_t token[2], head[2];   // strides
    uint8_t* codes[2];
    float* scale[2];
    uint32_t heads, dim, units;
};

// Work within a block goes by tokens of a chunk (64 of 128 dimensions, 8 KiB of codes), in pieces of
// four tokens x eight dimensions, one a thread.
__device__ inline uint32_t chunk_tokens(uint32_t units) { return units <= 2 ? 128 : units <= 4 ? 64 : 32; }

// A chunk's codes in LDS: the 256 bytes of a unit that 16 lanes load lie 272 apart,
// so that pieces of neighbouring dimensions and tokens meet other banks.
constexpr uint32_t PITCH = 272;
__device__ inline uint32_t padded_at(uint32_t byte) { return byte / 256 * PITCH + byte % 256; }

struct Piece4 {
    uint32_t t, d;   // first token (of the chunk) and dimension
    bool real;
    __device__ Piece4(uint32_t i, uint32_t tokens, uint32_t dim) {
        const uint32_t across = (dim + 7) / 8;
        t = i / across * 4;
        d = i % across * 8;
        real = t < tokens;
    }
};

// A workgroup writes the rows of one span for one head, keys or values: their
// largest magnitude first, then the codes.  A block of one chunk stays in
// registers in between.  Codes of chunks that hold new tokens alone (or nothing
// yet behind them) are put together in LDS and stored by 16-byte pieces; where
// older tokens share the chunk, as in a decoding step, each goes to its own place.
//
// Bound by HBM: eight prompts of 2048 tokens, 8 heads of 128 dimensions in bf16, 24 us,
// 4.2 TB/s of what it reads and writes (38 with a second pass over the rows and bytes
// into LDS); 64 sequences' newest tokens 7 us, a chain of five loads.
template <typename T>
__global__ __launch_bounds__(THREADS) void cache_write_kernel(WriteArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_codes[32 * PITCH];
    __shared__ uint32_t s_max[THREADS / 64];
    Span p;
    if (!p.find(a.seqs, blockIdx.x, threadIdx.x & 63) || p.bad) return;
    const uint32_t which = blockIdx.z, h = blockIdx.y, block = a.seqs.block, dim = a.dim;
    const uint64_t cell = (uint64_t)p.page * a.heads + h, stride = a.token[which];
    const T* x = reinterpret_cast<const T*>(a.x[which]) + h * a.head[which];
    const float was = a.scale[which][cell];
    const uint32_t chunk = umin(chunk_tokens(a.units), block), first = p.lo / chunk * chunk;

    // a piece's tokens, zeros where they are not new
    auto load = [&](uint32_t begin, const Piece4& c, Piece<T> (&v)[4]) {
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t t = begin + c.t + j;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j].set(i, 0.0f);
            if (c.real && t >= p.lo && t < p.hi) v[j].load(x + (uint64_t)(p.row + t - p.lo) * stride + c.d, dim - c.d);
        }
    };
    Piece<T> v[4];
    uint32_t amax = 0;
    for (uint32_t begin = first; begin < p.hi; begin += chunk) {
        load(begin, Piece4(threadIdx.x, chunk, dim), v);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = umax(amax, __float_as_uint(v[j][e]) & ABS_MASK);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) amax = umax(amax, (uint32_t)__shfl_xor((int)amax, o));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x / 64] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) amax = umax(amax, s_max[i]);
    const float need = amax >= INF_BITS ? __uint_as_float(0x7fc00000u) : __uint_as_float(amax) / 127.0f;
    const bool kept = p.lo > 0;
    float scale = need;
    if (kept && need <= was) scale = was;
    if (kept && need > was) scale = fmaxf(need, 1.25f * was);
    if (kept && !(was == was)) scale = was;
    if (threadIdx.x == 0) a.scale[which][cell] = scale;
    Step step;
    step.set(scale);

    const uint32_t tile_bytes = a.units * UNIT_BYTES;
    uint8_t* out = a.codes[which] + cell * (block / TILE_TOKENS) * tile_bytes;
    if (kept && __float_as_uint(scale) != __float_as_uint(was)) {
        // the older codes' tiles, rounded again: codes of 8 bits by scales of 24 give quotients that never lie
        // nearer to half a step than 64 bits tell
        u32x4* mem = reinterpret_cast<u32x4*>(out);
        const uint32_t n = (p.lo + TILE_TOKENS - 1) / TILE_TOKENS * tile_bytes / 16;
        for (uint32_t i = threadIdx.x; i < n; i += THREADS) {
            u32x4 w = mem[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t r = 0;
#pragma unroll
                for (int b = 0; b < 32; b += 8) {
                    const double q = (double)(int8_t)(w[j] >> b) * (double)was / (double)scale;
                    const int n = step.inv > 0.0f ? (int)fmin(fmax(rint(q), -127.0), 127.0) : 0;
                    r |= (uint32_t)(n & 255) << b;
                }
                w[j] = r;
            }
            mem[i] = w;
        }
        __syncthreads();   // new codes go over these
    }

    for (uint32_t begin = first; begin < p.hi; begin += chunk) {
        const Piece4 c(threadIdx.x, chunk, dim);
        if (block > chunk) load(begin, c, v);
        u32x2 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = v[j][e];
            q[j] = codes_of(step, f);
        }
        uint8_t* mem = out + begin / TILE_TOKENS * tile_bytes;
        const uint32_t unit = (c.t / TILE_TOKENS * a.units + c.d / 32) * UNIT_BYTES, t = c.t % TILE_TOKENS, d = c.d % 32;
        if (begin < p.lo) {
            if (!c.real) continue;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                if (begin + c.t + j < p.lo || begin + c.t + j >= p.hi) continue;
                if (which == 0) {
                    *reinterpret_cast<u32x2*>(mem + unit + key_byte(t + j, d)) = q[j];
                } else {
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        mem[unit + value_byte(t + j, d + e)] = (uint8_t)(q[j][e / 4] >> (8 * (e % 4)));
                }
            }
            continue;
        }
        // dimensions past the head's and tokens past the last are zeros
        const uint32_t bytes = chunk / TILE_TOKENS * tile_bytes;
        if (dim <= (a.units - 1) * 32 + 24) {
            for (uint32_t i = threadIdx.x; i < bytes / 16; i += THREADS)
                *reinterpret_cast<u32x4*>(s_codes + padded_at(i * 16)) = u32x4{0, 0, 0, 0};
            __syncthreads();
        }
        if (c.real) {
            if (which == 0) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    *reinterpret_cast<u32x2*>(s_codes + padded_at(unit + key_byte(t + j, d))) = q[j];
            } else {
                // four tokens' codes of a dimension are a word
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t a0 = __builtin_amdgcn_perm(q[1][i], q[0][i], 0x05010400u);   // 0 and 1 of tokens 0, 1
                    const uint32_t a1 = __builtin_amdgcn_perm(q[1][i], q[0][i], 0x07030602u);   // 2 and 3
                    const uint32_t b0 = __builtin_amdgcn_perm(q[3][i], q[2][i], 0x05010400u);
                    const uint32_t b1 = __builtin_amdgcn_perm(q[3][i], q[2][i], 0x07030602u);
                    const uint32_t r[4] = {__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                                           __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint32_t*>(s_codes + padded_at(unit + value_byte(t, d + 4 * i + e))) = r[e];
                }
            }
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < bytes / 16; i += THREADS)
            reinterpret_cast<u32x4*>(mem)[i] = *reinterpret_cast<const u32x4*>(s_codes + padded_at(i * 16));
        if (block > chunk) __syncthreads();
    }
}

// `items` workgroups along x have a span each.
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

// A workgroup reads the rows of one span for one head, keys or values, chunk by
// chunk through LDS, and writes whole rows.  Bound by HBM: the prompts above 18 us, 5.6 TB/s.
template <typename T>
__global__ __launch_bounds__(THREADS) void cache_read_kernel(ReadArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t s_codes[32 * PITCH];
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
    if (!p.find(a.seqs, blockIdx.x, threadIdx.x & 63)) return;
    if (p.bad) {
        for (uint32_t i = 0; i < p.hi - p.lo; ++i)
            put_row(out + (uint64_t)(p.row + i) * stride, a.dim, __uint_as_float(0x7fc00000u));
        return;
    }
    const uint64_t cell = (uint64_t)p.page * a.heads + h;
    const uint32_t tile_bytes = a.units * UNIT_BYTES, chunk = umin(chunk_tokens(a.units), block);
    const uint8_t* in = a.codes[which] + cell * (block / TILE_TOKENS) * tile_bytes;
    const float scale = a.scale[which][cell];
    const Piece4 c(threadIdx.x, chunk, a.dim);
    const uint32_t unit = (c.t / TILE_TOKENS * a.units + c.d / 32) * UNIT_BYTES, t = c.t % TILE_TOKENS, d = c.d % 32;
    for (uint32_t begin = p.lo / chunk * chunk; begin < p.hi; begin += chunk) {
        const u32x4* mem = reinterpret_cast<const u32x4*>(in + begin / TILE_TOKENS * tile_bytes);
        for (uint32_t i = threadIdx.x; i < chunk / TILE_TOKENS * tile_bytes / 16; i += THREADS)
            *reinterpret_cast<u32x4*>(s_codes + padded_at(i * 16)) = mem[i];
        __syncthreads();
        if (c.real) {
            u32x2 q[4];
            if (which == 0) {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
                    q[j] = *reinterpret_cast<const u32x2*>(s_codes + padded_at(unit + key_byte(t + j, d)));
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[e] = *reinterpret_cast<const uint32_t*>(s_codes + padded_at(unit + value_byte(t, d + 4 * i + e)));
                    const uint32_t a0 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u);
                    const uint32_t a1 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
                    const uint32_t b0 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
                    const uint32_t b1 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
                    q[0][i] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
                    q[1][i] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
                    q[2][i] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
                    q[3][i] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t at = begin + c.t + j;
                Piece<T> v;
#pragma unroll
                for (int e = 0; e < 8; ++e) v.set(e, product((float)(int8_t)(q[j][e / 4] >> (8 * (e % 4))), scale));
                if (at >= p.lo && at < p.hi) v.store(out + (uint64_t)(p.row + at - p.lo) * stride + c.d, a.dim - c.d);
            }
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
    const uint32_t more = s.starts ? s.tokens / 256 < 64 ? s.tokens / 256 + 1 : 64 : (s.seqs + 63) / 64;
    const ReadArgs a = {seqs_of(c, s), {static_cast<const uint8_t*>(c.k), static_cast<const uint8_t*>(c.v)},
                        {c.k_scale, c.v_scale}, {k, v}, c.heads, c.dim, padded_dim(c.dim) / 32, items, fill};
    return with_float_type(type, [&](auto t) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(cache_read_kernel<decltype(t)>), dim3(items + more, c.heads, 2), dim3(THREADS),
                           0, static_cast<hipStream_t>(stream), a);
        return launched();
    });
}

}  // namespace lecb
