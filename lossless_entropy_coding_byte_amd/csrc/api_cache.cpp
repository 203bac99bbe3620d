// C ABI of the 8-bit cache of keys and values and of the attention over it:
// argument checks, then one launch function each.  No allocation, no
// synchronisation.
#include <cmath>

#include "cache.hpp"

using namespace lecb;

namespace {

bool aligned(const void* p, uint64_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool geometry_ok(const lecb_cache_q8& c) {
    return c.blocks >= 1 && c.blocks < (1ull << 31) && c.heads >= 1 && c.heads <= 65535 && c.dim >= 1 && c.dim <= 256 &&
           valid_block(c.block);
}
bool cache_ok(const lecb_cache_q8* c) {
    return c && geometry_ok(*c) && c->k && c->v && aligned(c->k, 16) && aligned(c->v, 16) && c->k_scale && c->v_scale &&
           aligned(c->k_scale, 4) && aligned(c->v_scale, 4);
}
// OK, or the error
int seqs_status(const lecb_cache_q8& c, const lecb_cache_seqs* s) {
    if (!s) return LECB_ERR_INVALID_ARG;
    if (s->seqs >= (1u << 20) || s->tokens >= (1u << 27) || (uint64_t)s->width * c.block >= (1ull << 30))
        return LECB_ERR_TOO_LARGE;
    if (s->tokens == 0) return LECB_OK;
    if (!s->starts && s->tokens != s->seqs) return LECB_ERR_INVALID_ARG;
    if (s->seqs && (!s->table || !s->lengths || s->width < 1 || s->table_stride < s->width || !aligned(s->table, 4) ||
                    !aligned(s->lengths, 4)))
        return LECB_ERR_INVALID_ARG;
    return aligned(s->starts, 4) ? LECB_OK : LECB_ERR_INVALID_ARG;
}
// Each workgroup of the attention looks through all sequences for its own rows: 52 ms for 8192 sequences of a row, 32
// heads to 8, with starts (2^31.3 here), four times that with twice the sequences.  A sequence and head has up to four
// workgroups of 16 rows or one to 128.
bool search_ok(uint64_t seqs, uint64_t tokens, uint64_t heads, uint64_t cache_heads, uint64_t rows) {
    return seqs * (5 * seqs * cache_heads + tokens * heads / rows) < (1ull << 37);
}
uint64_t rows_of(int type, uint32_t dim) { return type == LECB_F32 && dim > 128 ? 16 : 128; }   // of a workgroup, of many
bool tensor_ok(const void* p, int type) { return p && aligned(p, elem_bytes(type)); }

}  // namespace

extern "C" {

uint64_t lecb_cache_q8_bytes(uint64_t blocks, uint32_t heads, uint32_t dim, uint32_t block) {
    const lecb_cache_q8 c = {nullptr, nullptr, nullptr, nullptr, blocks, heads, dim, block};
    return geometry_ok(c) ? blocks * heads * block * padded_dim(dim) : 0;
}

int lecb_cache_write_q8(const lecb_cache_q8* cache, const lecb_cache_seqs* seqs, const void* d_k, const void* d_v,
                        int type, uint64_t k_token_stride, uint64_t k_head_stride, uint64_t v_token_stride,
                        uint64_t v_head_stride, void* stream) {
    if (!cache_ok(cache) || !float_type(type)) return LECB_ERR_INVALID_ARG;
    if (const int rc = seqs_status(*cache, seqs)) return rc;
    if (seqs->tokens == 0 || seqs->seqs == 0) return LECB_OK;
    if (!tensor_ok(d_k, type) || !tensor_ok(d_v, type)) return LECB_ERR_INVALID_ARG;
    return launch_cache_write_q8(*cache, *seqs, d_k, d_v, type, k_token_stride, k_head_stride, v_token_stride,
                                 v_head_stride, stream);
}

int lecb_cache_read_q8(const lecb_cache_q8* cache, const lecb_cache_seqs* seqs, void* d_k, void* d_v, int type,
                       int fill, void* stream) {
    if (!cache_ok(cache) || !float_type(type) || (fill != 0 && fill != 1)) return LECB_ERR_INVALID_ARG;
    if (const int rc = seqs_status(*cache, seqs)) return rc;
    if (seqs->tokens == 0) return LECB_OK;
    if (seqs->seqs == 0 || !tensor_ok(d_k, type) || !tensor_ok(d_v, type)) return LECB_ERR_INVALID_ARG;
    return launch_cache_read_q8(*cache, *seqs, d_k, d_v, type, fill, stream);
}

uint64_t lecb_attention_q8_workspace_bytes(const lecb_cache_q8* cache, uint32_t seqs, uint32_t tokens, uint32_t width,
                                           uint32_t heads) {
    if (!cache || !geometry_ok(*cache) || heads < 1 || heads % cache->heads || seqs >= (1u << 20) ||
        tokens >= (1u << 27) || (uint64_t)width * cache->block >= (1ull << 30) || !seqs || !tokens ||
        !search_ok(seqs, tokens, heads, cache->heads, 128))
        return 0;
    return attention_q8_workspace(*cache, seqs, tokens, width, heads);
}

int lecb_attention_q8(const void* d_q, uint64_t q_token_stride, uint64_t q_head_stride, int type, uint32_t heads,
                      const lecb_cache_q8* cache, const lecb_cache_seqs* seqs, float scale, int causal,
                      uint32_t window, void* d_out, uint64_t out_token_stride, uint64_t out_head_stride, int fill,
                      void* d_ws, uint64_t ws_bytes, void* stream) {
    if (!cache_ok(cache) || !float_type(type) || heads < 1 || heads % cache->heads || !std::isfinite(scale * LOG2_E) ||
        (causal != 0 && causal != 1) || (fill != 0 && fill != 1) || (window && !causal) || window >= (1u << 31))
        return LECB_ERR_INVALID_ARG;
    if (const int rc = seqs_status(*cache, seqs)) return rc;
    if (seqs->tokens == 0) return LECB_OK;
    if ((uint64_t)seqs->tokens * heads >= (1ull << 27) || (uint64_t)seqs->seqs * cache->heads >= (1ull << 22) ||
        !search_ok(seqs->seqs, seqs->tokens, heads, cache->heads, rows_of(type, cache->dim)))
        return LECB_ERR_TOO_LARGE;
    if (seqs->seqs == 0 || !tensor_ok(d_q, type) || !tensor_ok(d_out, type) || out_head_stride < cache->dim ||
        out_token_stride < cache->dim)
        return LECB_ERR_INVALID_ARG;
    const uint64_t need = attention_q8_workspace(*cache, seqs->seqs, seqs->tokens, seqs->width, heads);
    if (need && (!d_ws || !aligned(d_ws, 16))) return LECB_ERR_INVALID_ARG;
    if (ws_bytes < need) return LECB_ERR_WORKSPACE;
    return launch_attention_q8({*cache, *seqs, d_q, d_out, type, q_token_stride, q_head_stride, out_token_stride,
                                out_head_stride, heads, scale, causal, window, fill, d_ws},
                               stream);
}

}  // extern "C"
