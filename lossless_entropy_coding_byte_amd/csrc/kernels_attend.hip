// Attention over the 8-bit cache: the kernels of both forms, what joins the parts
// of rows that were split, and the launches.  lecb.h states the formula.
#include "attend_few.hpp"
#include "attend_many.hpp"

namespace lecb {

namespace {

constexpr uint32_t FAR = 1u << 30;   // no row of the table holds more tokens
constexpr int WAVES = 4;
constexpr int THREADS = 64 * WAVES;

// Rows of 192 dimensions of 24 bits do not fit the registers of the form for many.
template <typename T, int U>
constexpr bool HAS_MANY = sizeof(T) == 2 || U < 6;

// A workgroup takes one item.  Those of the first launch without one see to the
// rows of no sequence.  16-bit rows of 128 dimensions are held to four workgroups a compute unit: with three, each
// finds its item while fewer others load (1024 sequences of 512 tokens 376 us, with four 334; one of 32768 with 64 rows 50 and 48).
template <typename T, int U>
__global__ __launch_bounds__(THREADS, U * sizeof(T) <= 8 ? 4 : U * sizeof(T) <= 16 ? 2 : 1) void attend_few_kernel(AttendArgs a) {
    __shared__ __attribute__((aligned(16))) FewMemory<T, U, WAVES> memory;
    const uint32_t h = blockIdx.x % a.heads, w = blockIdx.x / a.heads;
    Item it;
    if (find_item<FEW_ROWS, false>(a, w, threadIdx.x & 63, it))
        attend_few<T, U, WAVES>(a, it, h, memory);
    else if (a.fill)
        fill_rows<T>(a, (w - it.slot) * a.heads + h, (gridDim.x / a.heads - it.slot) * a.heads);
}

template <typename T, int U>
__global__ __launch_bounds__((2 * MANY_ROWS<T, U>), U * sizeof(T) <= 8 ? 2 : 1) void attend_many_kernel(AttendArgs a) {
    __shared__ __attribute__((aligned(16))) ManyMemory<T, U> memory;
    const uint32_t h = blockIdx.x % a.heads, w = blockIdx.x / a.heads;
    Item it;
    if (find_item<MANY_ROWS<T, U>, false>(a, w, threadIdx.x & 63, it))
        attend_many<T, U>(a, it, h, memory);
    else if (a.fill)
        fill_rows<T>(a, (w - it.slot) * a.heads + h, (gridDim.x / a.heads - it.slot) * a.heads);
}

// Rows whose tiles were split: SHARES groups of threads add up a row's parts, each
// in their order, and then their sums.
template <typename T, int U, int ROWS, bool WHOLE>
__device__ inline void join(const AttendArgs& a, const Item& it, uint32_t h, uint32_t z, uint32_t zs, float* memory) {
    constexpr int LANES = 8 * U, GROUPS = THREADS / LANES, SHARES = WHOLE ? GROUPS : 1, EACH = GROUPS / SHARES;
    constexpr int PITCH = 32 * U + 4;
    Work k;
    if (!work_of<ROWS>(a, it, h, k) || k.slot + (uint64_t)(k.parts - 1) * a.heads >= form_of<ROWS>(a).slots) return;
    const uint32_t group = threadIdx.x / LANES, d = threadIdx.x % LANES * 4, share = group % SHARES;
    const uint64_t step = (uint64_t)a.heads * ROWS * PITCH;
    for (uint32_t row0 = z * EACH; row0 < k.have; row0 += zs * EACH) {
        const uint32_t row = row0 + group / SHARES;
        float ref = inf(), l = 0.0f;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        if (group < GROUPS && row < k.have) {
            const float* ws = form_of<ROWS>(a).ws + ((uint64_t)k.slot * ROWS + row) * PITCH;
#pragma unroll 4
            for (uint32_t p = share; p < k.parts; p += SHARES) {
                const float* w = ws + p * step;
                const float r = w[0], next = fminf(ref, r), l2 = w[1];
                const f32x4 x = *reinterpret_cast<const f32x4*>(w + 4 + d);
                const float was = ref == next ? 1.0f : root_of(next - ref), is = r == next ? 1.0f : root_of(next - r);
                v = v * (was * was) + x * (is * is);
                l = l * was * was + l2 * is * is;
                ref = next;
            }
        }
        if (SHARES > 1) {
            float* s_sum = memory;                   // [SHARES][32 U]
            float* s_ref = memory + SHARES * 32 * U;
            float* s_l = s_ref + SHARES;
            if (group < GROUPS) {
                *reinterpret_cast<f32x4*>(s_sum + share * 32 * U + d) = v;
                if (d == 0) {
                    s_ref[share] = ref;
                    s_l[share] = l;
                }
            }
            __syncthreads();
            if (share == 0) {
                float least = s_ref[0];
#pragma unroll
                for (int j = 1; j < SHARES; ++j) least = fminf(least, s_ref[j]);
                v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                l = 0.0f;
#pragma unroll
                for (int j = 0; j < SHARES; ++j) {
                    const float root = s_ref[j] == least ? 1.0f : root_of(least - s_ref[j]);
                    v += *reinterpret_cast<const f32x4*>(s_sum + j * 32 * U + d) * (root * root);
                    l += s_l[j] * root * root;
                }
            }
            __syncthreads();
        }
        if (share == 0 && group < GROUPS && row < k.have) {
            const float up = l == 0.0f ? 0.0f : OUT / l;
            const T o[4] = {(T)(v[0] * up), (T)(v[1] * up), (T)(v[2] * up), (T)(v[3] * up)};
            put_four(a, k, h, k.r0 + row, d, o);
        }
    }
}

// Few rows have many parts: a workgroup joins one row.  Many rows have few: as many
// rows at a time as there are groups of threads.
template <typename T, int U, bool MANY>
__global__ __launch_bounds__(THREADS) void attend_join_kernel(AttendArgs a, uint32_t few_items) {
    __shared__ __attribute__((aligned(16))) float memory[THREADS * 4 + 2 * THREADS / (8 * U)];
    const uint32_t lane = threadIdx.x & 63;
    Item it;
    if (blockIdx.x < few_items) {
        if (find_item<FEW_ROWS, true>(a, blockIdx.x, lane, it))
            join<T, U, FEW_ROWS, true>(a, it, blockIdx.y, blockIdx.z, gridDim.z, memory);
    } else if (MANY && find_item<MANY_ROWS<T, U>, true>(a, blockIdx.x - few_items, lane, it)) {
        join<T, U, MANY_ROWS<T, U>, false>(a, it, blockIdx.y, blockIdx.z, gridDim.z, memory);
    }
}

// What a form's work may come to, whatever the lengths are.  Workgroups wished for
// are as many as the GPU holds at once; a part has `shortest` tiles at least: one for
// each wave of the form for few rows where a tile is short work (one token after 1000 in 128
// dimensions 10.4 us, with two 11.2), two where it is not (8 sequences with windows of 4096 in
// 256 dimensions 16.8 us, with one 19.3).
struct Shape {
    uint64_t items, joins;   // for each head: workgroups, rows that are split
    uint64_t slots;          // of all heads
    uint32_t target, shortest;
};
// rows: of a workgroup.
Shape shape_of(uint64_t rows, uint32_t dim, uint32_t heads, uint32_t group, uint32_t block, uint64_t seqs, uint64_t tokens, uint64_t width,
               uint64_t few) {
    const bool many = rows != FEW_ROWS;
    Shape s;
    s.target = (uint32_t)((many ? rows == 128 ? 2 : 1 : 4) * device_cu_count());
    s.shortest = many ? 16 : dim <= 128 ? 4 : 8;
    // a sequence's rows, rounded up; none has more than `few` in the form for few
    uint64_t most = tokens * group / rows + seqs;
    if (tokens * tiles_of(group, rows) < most) most = tokens * tiles_of(group, rows);
    if (!many && seqs * tiles_of(few, rows) < most) most = seqs * tiles_of(few, rows);
    const uint64_t parts = tiles_of(width * block / TILE_TOKENS + 2, s.shortest);
    const bool split = parts > 1;
    s.items = split ? s.target / heads < most * (parts - 1) ? most + s.target / heads : most * parts : most;
    s.items += 1;   // one without an item, for the rows of no sequence
    s.joins = split ? s.target / heads < most ? s.target / heads : most : 0;
    s.slots = split ? 2ull * s.target : 0;
    if (split && most * heads * parts < s.slots) s.slots = most * heads * parts;
    if (!split) s.shortest = 0x7ffffffeu;
    return s;
}
uint64_t bytes_of(const Shape& s, uint64_t rows, uint32_t dim) {
    return s.slots * rows * (padded_dim(dim) + 4) * sizeof(float);
}

// Rows of a sequence up to which the form for few takes it.  Both forms, us, heads
// of 128 dimensions in bf16: 16 sequences of 8192 tokens with 64 rows each 131 and 156,
// one of 32768 48 and 52, 16 of 1024 34 and 36; with 128 rows 206 and 162 (8192), 66 and 55
// (32768), 35 and 41 (1024), with 512 655 and 317, 186 and 96, 104 and 62; dimensions of 64 and 256 and
// 32 bits cross between 64 and 256 rows too.  Neither the heads of the cache nor the lengths enter: with
// one head or short sequences the form for many leaves compute units idle that the other would use.  Each form takes a launch, 4 to 5 us where it finds nothing to
// do: a call of few rows in all goes by the form for few alone, one sequence by one of them.
uint32_t few_most(int type, uint32_t dim, uint64_t rows, uint64_t seqs) {
    if ((type == LECB_F32 && dim > 128) || rows <= (seqs > 1 ? 256 : 64)) return 0x7fffffffu;
    return seqs > 1 ? 64 : 0;
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

template <typename T, int U>
int launch(AttendArgs a, const Shape* shape, bool few, bool many, hipStream_t st) {
    uint32_t joins[2] = {0, 0};
    if constexpr (HAS_MANY<T, U>)
        if (many) {
            hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_many_kernel<T, U>), dim3((uint32_t)(shape[1].items * a.heads)),
                               dim3(2 * MANY_ROWS<T, U>), 0, st, a);
            joins[1] = (uint32_t)shape[1].joins;
            a.fill = 0;
        }
    if (few) {
        hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_few_kernel<T, U>), dim3((uint32_t)(shape[0].items * a.heads)),
                           dim3(THREADS), 0, st, a);
        joins[0] = (uint32_t)shape[0].joins;
    }
    const uint32_t all = joins[0] + joins[1];
    if (all) {
        // as many workgroups to the same rows as make about eight for each compute unit
        const uint32_t most = a.seqs.starts || a.group > FEW_ROWS ? FEW_ROWS : a.group;
        uint32_t z = 8u * (uint32_t)device_cu_count() / (all * a.heads);
        z = z < 1 ? 1 : z < most ? z : most;
        if (joins[1])
            hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_join_kernel<T, U, HAS_MANY<T, U>>), dim3(all, a.heads, z), dim3(THREADS),
                               0, st, a, joins[0]);
        else
            hipLaunchKernelGGL(HIP_KERNEL_NAME(attend_join_kernel<T, U, false>), dim3(all, a.heads, z), dim3(THREADS), 0, st,
                               a, joins[0]);
    }
    return launched();
}

}  // namespace

uint64_t attention_q8_workspace(const lecb_cache_q8& c, uint64_t seqs, uint64_t tokens, uint64_t width, uint32_t heads) {
    // for every type, and with starts or without
    const uint32_t group = heads / c.heads;
    auto bytes = [&](uint64_t rows) {
        return bytes_of(shape_of(rows, c.dim, c.heads, group, c.block, seqs, tokens, width, few_most(LECB_F32, c.dim, tokens * group, seqs)),
                        rows, c.dim);
    };
    // the form for many, where a sequence that had all rows would go by it in any type
    const bool any = tokens * group > few_most(LECB_BF16, c.dim, tokens * group, seqs);
    const uint64_t many = any ? bytes(128) : 0, more = any ? bytes(256) : 0;
    return bytes(FEW_ROWS) + (many > more ? many : more);
}

int launch_attention_q8(const AttentionQ8& x, void* stream) {
    const uint32_t group = x.heads / x.cache.heads;
    const uint64_t rows = (uint64_t)x.seqs.tokens * group, longest = x.seqs.starts ? rows : group;   // a sequence may have all of them
    const uint32_t most = few_most(x.type, x.cache.dim, rows, x.seqs.seqs);
    const bool many = longest > most, few = most > 0 && (!many || x.seqs.starts);
    AttendArgs a = {seqs_of(x.cache, x.seqs), x.q, x.out, static_cast<const uint8_t*>(x.cache.k),
                    static_cast<const uint8_t*>(x.cache.v), x.cache.k_scale, x.cache.v_scale, x.q_token, x.q_head, x.out_token,
                    x.out_head, x.cache.heads, group, x.cache.dim, x.window < FAR ? x.window : FAR, x.causal, x.fill,
                    x.scale * LOG2_E, most, {}};
    return with_float_type(x.type, [&](auto t) {
        typedef decltype(t) T;
        return with_units(x.cache.dim, [&](auto units) {
            constexpr int U = decltype(units)::value;
            constexpr uint64_t ROWS[2] = {FEW_ROWS, MANY_ROWS<T, U>};
            Shape shape[2];
            float* ws = static_cast<float*>(x.ws);
            for (int i = 0; i < 2; ++i) {
                shape[i] = shape_of(ROWS[i], a.dim, a.heads, group, x.cache.block, x.seqs.seqs, x.seqs.tokens, x.seqs.width, most);
                a.form[i] = {ws, shape[i].target, shape[i].shortest, (uint32_t)shape[i].slots};
                ws += bytes_of(shape[i], ROWS[i], a.dim) / sizeof(float);
            }
            return launch<T, U>(a, shape, few, many, static_cast<hipStream_t>(stream));
        });
    });
}

}  // namespace lecb
