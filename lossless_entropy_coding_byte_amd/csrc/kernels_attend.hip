// Attention over the 8-bit cache: the form for few rows, and what joins the
// parts of rows that were split.  lecb.h states the formula.
#include "attend.hpp"

namespace lecb {

namespace {

constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;

__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// A tile of 32 tokens, in registers as it lies.
template <int U>
struct Tile {
    u32x4 k[U], v[U];
    float k_scale, v_scale;
    __device__ void load(const AttendArgs& a, uint32_t page, uint32_t t, uint32_t shift, uint32_t h, uint32_t lane) {
        const bool none = page >= a.seqs.blocks;
        const uint64_t cell = (uint64_t)(none ? 0 : page) * a.heads + h;
        const uint64_t at = ((cell << shift) + (t & ((1u << shift) - 1))) * (U * UNIT_BYTES) + lane * 16;
#pragma unroll
        for (int u = 0; u < U; ++u)
            k[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.k + at + u * UNIT_BYTES));
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.v + at + u * UNIT_BYTES));
        const float ks = a.k_scale[cell];
        k_scale = none ? __uint_as_float(0x7fc00000u) : ks;
        v_scale = a.v_scale[cell];
    }
};

// Few rows: a workgroup takes 16 NT rows of one head over a part of the tiles,
// its waves tile by tile in turn, each with a softmax of its own; their sums are
// joined at the end.  Matrix instructions by 16 x 16 x 32, transposed: codes of
// 16 tokens (then of 16 dimensions of the values) times the rows, so that a row's
// scores stand in one lane of each 16, four tokens each, and are the second
// product's operand as they are; values are stored in that order of tokens.
// Neither codes nor scores go through LDS.
template <typename T, int U, int NT>
__global__ __launch_bounds__(THREADS) void attend_few_kernel(AttendArgs a) {
    constexpr int ROWS = 16 * NT, NQ = Parts<T>::Q, NP = Parts<T>::P;
    __shared__ __attribute__((aligned(16))) float s_sum[WAVES][ROWS][68];
    __shared__ float s_ref[WAVES][ROWS], s_l[WAVES][ROWS];
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const uint32_t w = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    Item it;
    if (!find_item<ROWS>(a, w, lane, it)) {
        if (a.fill) fill_rows<T>(a, (w - it.slot) * a.heads + h, (a.items - it.slot) * a.heads);
        return;
    }
    const uint32_t seq = uniform(it.seq), part = uniform(it.part), parts = uniform(it.parts);
    const uint32_t r0 = uniform(it.rows_at) * ROWS, slot = uniform(it.slot) * a.heads + h;
    const uint32_t n = uniform(a.seqs.count(seq)), len = uniform(a.seqs.length(seq)), begin = uniform(a.seqs.begin(seq));
    // starts that do not rise make more of either than there is room for
    if (r0 / ROWS >= (n * a.group + ROWS - 1) / ROWS || (parts > 1 && slot >= a.slots)) return;
    const uint32_t rows = n * a.group, have = rows - r0 < (uint32_t)ROWS ? rows - r0 : ROWS;
    T* out = reinterpret_cast<T*>(a.out) + (uint64_t)h * a.group * a.out_head;
    if (a.seqs.bad(len)) {
        for (uint32_t i = 0; i < have; ++i) {
            T* o = out + (uint64_t)(begin + (r0 + i) / a.group) * a.out_token + (r0 + i) % a.group * a.out_head;
            for (uint32_t d = threadIdx.x; d < a.dim; d += THREADS) o[d] = (T)__uint_as_float(0x7fc00000u);
        }
        return;
    }

    // rows: lane r of each 16 has row r of each 16, dimensions 32 u + 8 g and on
    f16x8 q[NT][U][NQ];
    float factor[NT];   // what takes a product of codes to a score
    int hi[NT], lo[NT];
    const int old = (int)len - (int)n;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const uint32_t i = r0 + 16 * c + r;
        const bool real = i < rows;
        const uint32_t token = real ? i / a.group : 0, head = real ? i % a.group : 0;
        const T* p = reinterpret_cast<const T*>(a.q) + (real ? (uint64_t)(begin + token) * a.q_token : 0) +
                     (uint64_t)(h * a.group + head) * a.q_head;
        Piece<T> x[U];
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t d = 32 * u + 8 * g, count = real && d < a.dim ? a.dim - d : 0;
            x[u].load(p + (count ? d : 0), count);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __float_as_uint(x[u][e]) & 0x7fffffffu;
                top = b > top ? b : top;
            }
        }
        uint32_t b = __shfl_xor(top, 16);
        top = b > top ? b : top;
        b = __shfl_xor(top, 32);
        top = b > top ? b : top;
        int lift = 0;
        if (Parts<T>::LIFT && top != 0) lift = 15 - __builtin_amdgcn_frexp_expf(__uint_as_float(top));
        factor[c] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : ldexpf(a.scale, -lift);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float f = Parts<T>::LIFT ? ldexpf(x[u][e], lift) : x[u][e];
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    q[c][u][j][e] = (_Float16)f;
                    f -= (float)q[c][u][j][e];
                }
            }
        hi[c] = a.causal ? old + (int)token : (int)len - 1;
        lo[c] = a.window ? old + (int)token - (int)a.window + 1 : 0;
    }

    // tiles: of the part, and those that some row sees; whole ones are seen by every row
    const int first_token = (int)(r0 / a.group), last_token = (int)((r0 + have - 1) / a.group);
    const int hi_least = a.causal ? old + first_token : (int)len - 1, hi_most = a.causal ? old + last_token : (int)len - 1;
    const int lo_least = a.window ? old + first_token - (int)a.window + 1 : 0;
    const int lo_most = a.window ? old + last_token - (int)a.window + 1 : 0;
    const uint64_t part_at = (uint64_t)uniform(it.first_tile) + (uint64_t)part * uniform(it.tiles);
    int from = (int)part_at, to = (int)uniform(it.last_tile);
    if (part_at + uniform(it.tiles) < (uint64_t)to) to = (int)(part_at + uniform(it.tiles));
    if (lo_least > 0 && lo_least / (int)TILE_TOKENS > from) from = lo_least / (int)TILE_TOKENS;
    const int seen = hi_most < 0 ? 0 : hi_most / (int)TILE_TOKENS + 1;
    if (seen < to) to = seen;

    f32x4 acc[NT][2 * U];
    float ref[NT], sum[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        ref[c] = inf();
        sum[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) acc[c][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const uint32_t shift = __builtin_ctz(a.seqs.block / TILE_TOKENS);

    auto compute = [&](int t, const Tile<U>& x) {
        f32x4 s[NT][2];
#pragma unroll
        for (int c = 0; c < NT; ++c) s[c][0] = s[c][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const f16x8 k = operand(x.k[u][2 * b], x.k[u][2 * b + 1]);
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
                        s[c][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[c][u][j], s[c][b], 0, 0, 0);
            }
        const int at = t * (int)TILE_TOKENS + 4 * (int)g;
        const bool whole = t * (int)TILE_TOKENS >= lo_most && t * (int)TILE_TOKENS + 31 <= hi_least;
        const float down = x.v_scale * P_DOWN, unit = scale_exponent(x.v_scale);
        f16x8 p[NT][NP];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const float f = factor[c] * x.k_scale;
            float v[8], most = -inf();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = s[c][i / 4][i % 4] * f;
                if (!whole) {
                    const int pos = at + i % 4 + i / 4 * 16;
                    v[i] = pos <= hi[c] && pos >= lo[c] ? v[i] : -inf();
                }
                most = fmaxf(most, v[i]);
            }
            most = fmaxf(most, __shfl_xor(most, 16));
            most = fmaxf(most, __shfl_xor(most, 32));
            const float next = fminf(ref[c], REF_TOP - (most + unit));
            if (__ballot(next < ref[c])) {
                const float down_by = next < ref[c] ? exp2_of(next - ref[c]) : 1.0f;
                sum[c] *= down_by;
#pragma unroll
                for (int i = 0; i < 2 * U; ++i) acc[c][i] *= down_by;
                ref[c] = next;
            }
            const float base = ref[c] == inf() ? 0.0f : ref[c];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = exp2_of(v[i] + base);
                sum[c] += v[i];
                v[i] = whole || v[i] != 0.0f ? v[i] * down : 0.0f;   // what is masked meets no scale
            }
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[c][j][i] = (_Float16)v[i];
                    v[i] -= (float)p[c][j][i];
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const f16x8 k = operand(x.v[u][2 * b], x.v[u][2 * b + 1]);
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        acc[c][2 * u + b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, p[c][j], acc[c][2 * u + b], 0, 0, 0);
            }
    };

    int t = from + (int)wave;
    if (t < to) {
        // the next tile's loads are in flight while one is worked on, its block's number one more ahead;
        // past the last tile the same one is asked for again
        Tile<U> x, y;
        auto page = [&](int i) { return uniform(a.seqs.page(seq, (uint32_t)(i < to ? i : t) >> shift)); };
        x.load(a, page(t), t, shift, h, lane);
        uint32_t ahead = page(t + WAVES);
        while (true) {
            int next = t + WAVES < to ? t + WAVES : t;
            y.load(a, ahead, next, shift, h, lane);
            ahead = page(t + 2 * WAVES);
            compute(t, x);
            t += WAVES;
            if (t >= to) break;
            next = t + WAVES < to ? t + WAVES : t;
            x.load(a, ahead, next, shift, h, lane);
            ahead = page(t + 2 * WAVES);
            compute(t, y);
            t += WAVES;
            if (t >= to) break;
        }
    }

    // the waves' sums, joined in their order
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        sum[c] += __shfl_xor(sum[c], 16);
        sum[c] += __shfl_xor(sum[c], 32);
        if (g == 0) {
            s_ref[wave][16 * c + r] = ref[c];
            s_l[wave][16 * c + r] = sum[c];
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        float least = s_ref[0][16 * c + r];
#pragma unroll
        for (int i = 1; i < WAVES; ++i) least = fminf(least, s_ref[i][16 * c + r]);
        const float down_by = ref[c] == least ? 1.0f : exp2_of(least - ref[c]);
#pragma unroll
        for (int i = 0; i < 2 * U; ++i) acc[c][i] *= down_by;
    }
    float* ws = a.ws + (uint64_t)slot * ROWS * (32 * U + 4);
#pragma unroll
    for (int d0 = 0; d0 < U; d0 += 2) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (2 * d0 + i < 2 * U)
                    *reinterpret_cast<f32x4*>(&s_sum[wave][16 * c + r][16 * i + 4 * g]) = acc[c][2 * d0 + i];
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < ROWS * 16; i += THREADS) {
            const uint32_t row = i / 16, d = i % 16 * 4;
            if (row >= have) break;
            f32x4 v = *reinterpret_cast<const f32x4*>(&s_sum[0][row][d]);
#pragma unroll
            for (int j = 1; j < WAVES; ++j) v += *reinterpret_cast<const f32x4*>(&s_sum[j][row][d]);
            float least = s_ref[0][row], l = 0.0f;
#pragma unroll
            for (int j = 1; j < WAVES; ++j) least = fminf(least, s_ref[j][row]);
#pragma unroll
            for (int j = 0; j < WAVES; ++j) l += s_l[j][row] * (s_ref[j][row] == least ? 1.0f : exp2_of(least - s_ref[j][row]));
            const uint32_t at = 32 * d0 + d;
            if (parts > 1) {
                if (at < 32 * U) *reinterpret_cast<f32x4*>(ws + row * (32 * U + 4) + 4 + at) = v;
                if (at == 0) {
                    ws[row * (32 * U + 4)] = least;
                    ws[row * (32 * U + 4) + 1] = l;
                }
            } else {
                const float up = l == 0.0f ? 0.0f : OUT / l;
                T* o = out + (uint64_t)(begin + (r0 + row) / a.group) * a.out_token + (r0 + row) % a.group * a.out_head + at;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at + j < a.dim) o[j] = (T)(v[j] * up);
            }
        }
        __syncthreads();
    }
}

// Rows whose tiles were split: a workgroup adds up one row's parts, in their
// order within each of 256 / (32 U / 4) shares.
template <typename T, int U, int ROWS>
__global__ __launch_bounds__(THREADS) void attend_join_kernel(AttendArgs a) {
    constexpr int LANES = 8 * U, SHARES = THREADS / LANES, PITCH = 32 * U + 4;
    __shared__ __attribute__((aligned(16))) float s_sum[SHARES][32 * U];
    __shared__ float s_ref[SHARES], s_l[SHARES];
    const uint32_t lane = threadIdx.x & 63, h = blockIdx.y;
    const uint32_t row = blockIdx.x;   // token * group + head of the group
    const uint32_t token = row / a.group;
    uint32_t seq = token;
    if (a.seqs.starts) {   // the last sequence that begins at the token or before and has rows there
        uint32_t s = 0, end = a.seqs.seqs;
        while (end - s > 1) {
            const uint32_t mid = (s + end) / 2;
            if (a.seqs.begin(mid) <= token)
                s = mid;
            else
                end = mid;
        }
        seq = s;
        if (token < a.seqs.begin(s) || token - a.seqs.begin(s) >= a.seqs.count(s)) return;
    }
    seq = uniform(seq);
    const uint32_t i = (token - a.seqs.begin(seq)) * a.group + row % a.group;   // of the sequence's rows
    // the slot of the sequence's first part
    const uint32_t part = part_tiles<ROWS>(a, lane);
    uint32_t slots = 0;
    for (uint32_t s0 = 0; s0 < seq; s0 += 64) {
        const Load l = load_of<ROWS>(a, s0 + lane < seq ? s0 + lane : a.seqs.seqs);
        const uint32_t parts = l.tiles > part ? (l.tiles + part - 1) / part : 1;
        slots = uniform(__shfl(scan32(parts > 1 ? l.rows * parts : 0, lane), 63) + slots);
    }
    const Load mine = load_of<ROWS>(a, seq);
    const uint32_t parts = mine.tiles > part ? (mine.tiles + part - 1) / part : 1;
    if (parts == 1) return;
    const uint64_t step = (uint64_t)a.heads * ROWS * PITCH, first = (uint64_t)(slots + i / ROWS * parts) * a.heads + h;
    if (first + (uint64_t)(parts - 1) * a.heads >= a.slots) return;   // as above
    const float* ws = a.ws + first * ROWS * PITCH + i % ROWS * PITCH;

    const uint32_t share = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
    float ref = inf(), l = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (share < SHARES) {
#pragma unroll 4
        for (uint32_t p = share; p < parts; p += SHARES) {
            const float* w = ws + p * step;
            const float next = fminf(ref, w[0]), l2 = w[1];
            const f32x4 x = *reinterpret_cast<const f32x4*>(w + 4 + d);
            const float was = ref == next ? 1.0f : exp2_of(next - ref), is = w[0] == next ? 1.0f : exp2_of(next - w[0]);
            v = v * was + x * is;
            l = l * was + l2 * is;
            ref = next;
        }
        *reinterpret_cast<f32x4*>(&s_sum[share][d]) = v;
        if (d == 0) {
            s_ref[share] = ref;
            s_l[share] = l;
        }
    }
    __syncthreads();
    if (share != 0) return;
    float least = s_ref[0];
#pragma unroll
    for (int j = 1; j < SHARES; ++j) least = fminf(least, s_ref[j]);
    v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    l = 0.0f;
#pragma unroll
    for (int j = 0; j < SHARES; ++j) {
        const float f = s_ref[j] == least ? 1.0f : exp2_of(least - s_ref[j]);
        v += *reinterpret_cast<const f32x4*>(&s_sum[j][d]) * f;
        l += s_l[j] * f;
    }
    const float up = l == 0.0f ? 0.0f : OUT / l;
    T* o = reinterpret_cast<T*>(a.out) + (uint64_t)token * a.out_token + (uint64_t)(h * a.group + row % a.group) * a.out_head + d;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (d + j < a.dim) o[j] = (T)(v[j] * up);
}

// Workgroups for the form for few rows: as many as the GPU holds at once.
constexpr uint64_t FEW_ROWS = 16, FEW_PER_CU = 4, SHORTEST = 8;

struct Shape {
    uint64_t items, slots;   // for each head; of all heads
    uint32_t target;
    bool split;
};
Shape shape_of(uint32_t heads, uint32_t group, uint32_t block, uint64_t seqs, uint64_t tokens, uint64_t width) {
    Shape s;
    s.target = (uint32_t)(FEW_PER_CU * device_cu_count());
    const uint64_t by_rows = tokens * group / FEW_ROWS + seqs, by_tokens = tokens * tiles_of(group, FEW_ROWS);
    const uint64_t most = by_rows < by_tokens ? by_rows : by_tokens;
    const uint64_t parts = tiles_of(width * block / TILE_TOKENS, SHORTEST);
    s.split = parts > 1 && tokens * group / FEW_ROWS * heads < s.target;
    s.items = most + (s.split ? s.target / heads : 0) + 1;
    s.slots = s.split ? 2ull * s.target : 0;
    if (s.split && most * heads * parts < s.slots) s.slots = most * heads * parts;
    return s;
}

template <typename F>
int with_units(uint32_t dim, F f) {
    switch (padded_dim(dim)) {
        case 64: return f(std::integral_constant<int, 2>());
        case 96: return f(std::integral_constant<int, 3>());
        case 128: return f(std::integral_constant<int, 4>());
        case 192: return f(std::integral_constant<int, 6>());
        default: return f(std::integral_constant<int, 8>());
    }
}

}  // namespace

uint64_t attention_q8_workspace(const lecb_cache_q8& c, uint64_t seqs, uint64_t tokens, uint64_t width, uint32_t heads) {
    const Shape s = shape_of(c.heads, heads / c.heads, c.block, seqs, tokens, width);
    return s.slots * FEW_ROWS * (padded_dim(c.dim) + 4) * sizeof(float);
}

int launch_attention_q8(const AttentionQ8& x, void* stream) {
    const uint32_t group = x.heads / x.cache.heads;
    const Shape s = shape_of(x.cache.heads, group, x.cache.block, x.seqs.seqs, x.seqs.tokens, x.seqs.width);
    AttendArgs a = {seqs_of(x.cache, x.seqs), x.q, x.out, static_cast<const uint8_t*>(x.cache.k),
                    static_cast<const uint8_t*>(x.cache.v), x.cache.k_scale, x.cache.v_scale, static_cast<float*>(x.ws),
                    x.q_token, x.q_head, x.out_token, x.out_head, x.cache.heads, group, x.cache.dim, x.window, x.causal,
                    x.fill, x.scale * 1.44269504088896340736f, s.target, s.split ? (uint32_t)SHORTEST : 0x7fffffffu,
                    (uint32_t)s.items, (uint32_t)s.slots};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return with_float_type(x.type, [&](auto t) {
        typedef decltype(t) T;
        return with_units(x.cache.dim, [&](auto units) {
            constexpr int U = decltype(units)::value;
            hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_few_kernel<T, U, 1>), dim3((uint32_t)(s.items * a.heads)),
                               dim3(THREADS), 0, st, a);
            if (s.split)
                hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_join_kernel<T, U, (int)FEW_ROWS>),
                                   dim3(x.seqs.tokens * group, a.heads), dim3(THREADS), 0, st, a);
            return launched();
        });
    });
}

}  // namespace lecb
