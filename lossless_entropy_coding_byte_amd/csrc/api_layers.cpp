// C ABI of the operators of quantised layers: argument checks and sizes, then
// one launch function each.  No allocation, no synchronisation.
#include <cmath>

#include "layers.hpp"
#include "lecb.h"

using namespace lecb;

namespace {

constexpr uint64_t MAX_DIM = 1ull << 31;   // rows and columns below this: tile counts fit 32 bits

bool aligned(const void* p, uint64_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dims_ok(uint64_t n, uint64_t k) { return n && k && n < MAX_DIM && k < MAX_DIM; }
bool tensor_ok(const void* p, int type) { return p && aligned(p, elem_bytes(type)); }

}  // namespace

extern "C" {

uint64_t lecb_w4_tile_bytes(uint64_t n, uint64_t k) {
    return dims_ok(n, k) ? tiles_of(n, TILE_ROWS) * tiles_of(k, TILE_COLS) * TILE_BYTES : 0;
}

uint64_t lecb_w4_scale_count(uint64_t n, uint64_t k, uint32_t group) {
    return dims_ok(n, k) && valid_group(group)
               ? tiles_of(n, TILE_ROWS) * tiles_of(k, TILE_COLS) * (TILE_COLS / group) * TILE_ROWS
               : 0;
}

int lecb_quantize_w4(const void* d_w, int type, uint64_t w_stride, uint64_t n, uint64_t k, uint32_t group,
                     uint8_t* d_tiles, void* d_scales, int scale_type, void* stream) {
    if (!dims_ok(n, k) || !float_type(type) || !valid_group(group) || !scale_type_ok(scale_type) ||
        w_stride < k || !tensor_ok(d_w, type) || !d_tiles || !d_scales || !aligned(d_tiles, 16) ||
        !aligned(d_scales, 16))
        return LECB_ERR_INVALID_ARG;
    return launch_quantize_w4({d_w, type, w_stride, n, k, group, d_tiles, d_scales, scale_type}, stream);
}

int lecb_dequantize_w4(const uint8_t* d_tiles, const void* d_scales, int scale_type, uint32_t group, uint64_t n,
                       uint64_t k, void* d_out, int type, uint64_t out_stride, void* stream) {
    if (!dims_ok(n, k) || !float_type(type) || !valid_group(group) || !scale_type_ok(scale_type) ||
        out_stride < k || !tensor_ok(d_out, type) || !d_tiles || !d_scales || !aligned(d_tiles, 16) ||
        !aligned(d_scales, 16))
        return LECB_ERR_INVALID_ARG;
    return launch_dequantize_w4({d_tiles, d_scales, scale_type, group, n, k, d_out, type, out_stride}, stream);
}

int lecb_tile_w4(const uint8_t* d_rows, uint64_t n, uint64_t k, uint8_t* d_tiles, void* stream) {
    if (!dims_ok(n, k) || !d_rows || !d_tiles || !aligned(d_tiles, 16)) return LECB_ERR_INVALID_ARG;
    return launch_tile_w4(d_rows, d_tiles, n, k, stream);
}

int lecb_untile_w4(const uint8_t* d_tiles, uint64_t n, uint64_t k, uint8_t* d_rows, void* stream) {
    if (!dims_ok(n, k) || !d_rows || !d_tiles || !aligned(d_tiles, 16)) return LECB_ERR_INVALID_ARG;
    return launch_untile_w4(d_tiles, d_rows, n, k, stream);
}

int lecb_rmsnorm_q8(const void* d_x, uint64_t x_stride, const void* d_res, uint64_t res_stride,
                    const void* d_weight, int weight_type, int type, uint64_t rows, uint32_t cols, float eps,
                    void* d_h, uint64_t h_stride, int8_t* d_q, float* d_scale, int static_scale, void* stream) {
    if (!float_type(type) || !float_type(weight_type) || cols < 1 || cols > LECB_NORM_MAX_COLS ||
        !(eps > 0) || !std::isfinite(eps) || (static_scale != 0 && static_scale != 1))
        return LECB_ERR_INVALID_ARG;
    if (rows == 0) return LECB_OK;
    if (rows >= MAX_DIM) return LECB_ERR_TOO_LARGE;
    if (x_stride < cols || (d_res && res_stride < cols) || (d_h && h_stride < cols) || !tensor_ok(d_x, type) ||
        (d_res && !tensor_ok(d_res, type)) || (d_h && !tensor_ok(d_h, type)) ||
        !tensor_ok(d_weight, weight_type) || !d_q || !d_scale || !aligned(d_scale, 4))
        return LECB_ERR_INVALID_ARG;
    if (d_h && ((d_h == d_x && h_stride != x_stride) || (d_h == d_res && h_stride != res_stride)))
        return LECB_ERR_INVALID_ARG;
    return launch_rmsnorm_q8({d_x, x_stride, d_res, res_stride, d_weight, weight_type, type, rows, cols, eps, d_h,
                              h_stride, d_q, d_scale, static_scale},
                             stream);
}

int lecb_dequantize_q8(const int8_t* d_q, uint64_t rows, uint64_t cols, const float* d_scale, int scale_stride,
                       void* d_out, int type, void* stream) {
    if (!float_type(type) || (scale_stride != 0 && scale_stride != 1)) return LECB_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return LECB_OK;
    if (rows >= MAX_DIM || cols >= MAX_DIM || rows * cols >= (1ull << 35)) return LECB_ERR_TOO_LARGE;
    if (!d_q || !d_scale || !d_out || !aligned(d_q, 16) || !aligned(d_scale, 4) || !aligned(d_out, 16))
        return LECB_ERR_INVALID_ARG;
    return launch_dequantize_q8(d_q, rows, cols, d_scale, scale_stride, d_out, type, stream);
}

uint64_t lecb_matvec_w4_workspace_bytes(uint64_t m, uint64_t n, uint64_t k) {
    return dims_ok(n, k) && m < MAX_DIM ? matvec_w4_workspace(m, n, k) : 0;
}

int lecb_matvec_w4(const void* d_x, int x_type, uint64_t x_stride, const float* d_xscale, int xscale_stride,
                   uint64_t m, const uint8_t* d_tiles, const void* d_scales, int scale_type, uint32_t group,
                   uint64_t n, uint64_t k, void* d_y, int y_type, uint64_t y_stride, void* d_ws,
                   uint64_t ws_bytes, void* stream) {
    if (!dims_ok(n, k) || !valid_group(group) || !scale_type_ok(scale_type) || !float_type(y_type) ||
        (x_type != LECB_I8 && x_type != LECB_BF16 && x_type != LECB_F16) ||
        (d_xscale && (x_type != LECB_I8 || !aligned(d_xscale, 4))) || (xscale_stride != 0 && xscale_stride != 1))
        return LECB_ERR_INVALID_ARG;
    if (m == 0) return LECB_OK;
    if (m >= MAX_DIM) return LECB_ERR_TOO_LARGE;
    if (x_stride < k || y_stride < n || !tensor_ok(d_x, x_type) || !tensor_ok(d_y, y_type) || !d_tiles ||
        !d_scales || !aligned(d_tiles, 16) || !aligned(d_scales, 16))
        return LECB_ERR_INVALID_ARG;
    const uint64_t need = matvec_w4_workspace(m, n, k);
    if (need && (!d_ws || !aligned(d_ws, 16))) return LECB_ERR_INVALID_ARG;
    if (ws_bytes < need) return LECB_ERR_WORKSPACE;
    return launch_matvec_w4({d_x, x_type, x_stride, d_xscale, xscale_stride, m, d_tiles, d_scales, scale_type,
                             group, n, k, d_y, y_type, y_stride, d_ws},
                            stream);
}

}  // extern "C"
