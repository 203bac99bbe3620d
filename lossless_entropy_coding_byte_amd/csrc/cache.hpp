// Declarations shared by the 8-bit cache of keys and values and the attention
// over it: geometry, sequences, launches.
#pragma once

#include "layers.hpp"

namespace lecb {

// Codes stand in units of 32 tokens x 32 dimensions (lecb.h gives the order
// within a unit): 1 KiB, one 16-byte load of a wave, and a lane's 16 bytes are
// two matrix operands as they lie.  A tile is a head's units of 32 tokens.
constexpr uint32_t TILE_TOKENS = 32;
constexpr uint32_t UNIT_BYTES = 1024;

// Dimensions as they are stored: kernels are made for these five.
inline uint32_t padded_dim(uint32_t d) { return d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }
inline bool valid_block(uint32_t b) { return b == 32 || b == 64 || b == 128 || b == 256; }

int launch_cache_write_q8(const lecb_cache_q8& c, const lecb_cache_seqs& s, const void* k, const void* v, int type,
                          uint64_t k_token, uint64_t k_head, uint64_t v_token, uint64_t v_head, void* stream);
int launch_cache_read_q8(const lecb_cache_q8& c, const lecb_cache_seqs& s, void* k, void* v, int type, int fill,
                         void* stream);

constexpr float LOG2_E = 1.44269504088896340736f;   // the softmax is one of powers of two

struct AttentionQ8 {
    lecb_cache_q8 cache;
    lecb_cache_seqs seqs;
    const void* q;
    void* out;
    int type;
    uint64_t q_token, q_head, out_token, out_head;   // strides
    uint32_t heads;
    float scale;
    int causal;
    uint32_t window;   // 0: none
    int fill;
    void* ws;
};
uint64_t attention_q8_workspace(const lecb_cache_q8& c, uint64_t seqs, uint64_t tokens, uint64_t width, uint32_t heads);
int launch_attention_q8(const AttentionQ8& a, void* stream);

}  // namespace lecb

#if defined(__HIPCC__)
namespace lecb {

// The sequences of a call.  What they hold is only known here, so nothing is
// taken on trust: starts are kept within the rows, and a sequence whose length
// does not fit its row of the table is `bad`.
struct Seqs {
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* starts;   // NULL: one row each
    uint64_t stride;
    uint32_t seqs, width, tokens, block, blocks;

    __device__ uint32_t begin(uint32_t s) const {
        if (!starts) return s;
        const int32_t b = starts[s];
        return b < 0 ? 0u : (uint32_t)b < tokens ? (uint32_t)b : tokens;
    }
    __device__ uint32_t count(uint32_t s) const {
        if (!starts) return 1;
        const uint32_t b = begin(s), e = begin(s + 1);
        return e > b ? e - b : 0u;
    }
    __device__ uint32_t length(uint32_t s) const {
        const int32_t n = lengths[s];
        return n < 0 ? 0u : (uint32_t)n;
    }
    __device__ bool bad(uint32_t length) const { return length > width * block; }   // fits 32 bits: checked on the host
    // The cache's block that holds a sequence's block j; `blocks` and more: none does.
    __device__ uint32_t page(uint32_t s, uint32_t j) const {
        return j < width ? (uint32_t)table[(uint64_t)s * stride + j] : 0xffffffffu;
    }
    // The rows of no sequence are those before starts[0] and from starts[seqs] on.
    __device__ uint32_t outside(uint32_t* first) const {   // their number; `first`: where the second part begins
        if (!starts) return 0;
        const uint32_t b = begin(0), e = begin(seqs);
        *first = e > b ? e : b;
        return b + tokens - *first;
    }
};

inline Seqs seqs_of(const lecb_cache_q8& c, const lecb_cache_seqs& s) {
    return {s.table, s.lengths, s.starts, s.table_stride, s.seqs, s.width, s.tokens, c.block, (uint32_t)c.blocks};
}

}  // namespace lecb
#endif
