// wc_api_q4.cu -- the extern "C" boundary of the 4-bit streams, their products
// and the expert routing: argument checks and launches. Contracts are in
// include/wcodec.h.
#include <stdint.h>

#include "../../include/wcodec.h"
#include "wc_q4_core.cuh"

namespace {

constexpr uint32_t kStreamFlags = WC_Q4_ZEROS | WC_Q4_SCALES_FP16;
constexpr uint32_t kAllFlags = kStreamFlags | WC_Q4_X_FP16 | WC_Q4_Y_16BIT;

// Rows of x a matrix (of experts: on average) up to which wc_q4_gemv.cu is taken.
// Measured, it and wc_q4_gemm.cu, us: 14336 x 4096, 8 rows 15.7 and 17.3, 16 rows
// 19.6 and 17.6, 24 rows 34 and 18; 4096 x 14336, 16 rows 17.3 and 17.5; 1024 x
// 4096, 16 rows 6.8 and 7.8, 24 rows 10.6 and 8.0. Experts (16 of 4096 x 2048),
// whose rows come unevenly: 8 a matrix 35.5 and 33.3, 16 a matrix 43.7 and 33.9.
// The host knows their mean alone (64 of 2048 x 1024, mean 6): all with 6 rows 29
// and 37, half of the rows at one 112 and 41, all at one 211 and 15.
constexpr uint64_t kFewRows = 16;
constexpr uint64_t kFewRowsExperts = 6;

bool aligned(const void* p, uint32_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }

bool q4_shape_ok(uint64_t rows, uint64_t cols, uint32_t group) {
    return wc::q4_group_ok(group) && rows <= WC_Q4_MAX_ROWS && cols >= 1 && cols <= WC_Q4_MAX_COLS;
}

int check_stream(const void* d_stream, uint64_t stream_bytes, uint64_t rows, uint64_t cols,
                 uint32_t group, uint32_t flags) {
    if (!q4_shape_ok(rows, cols, group) || d_stream == nullptr || !aligned(d_stream, 16))
        return WC_ERR_INVALID_ARG;
    if (stream_bytes < wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags).total)
        return WC_ERR_CORRUPT_STREAM;
    return WC_OK;
}

int result(cudaError_t err) { return err == cudaSuccess ? WC_OK : WC_ERR_CUDA; }

uint32_t dtype_size(uint32_t dtype) { return dtype == WC_DTYPE_FP32 ? 4u : 2u; }

}  // namespace

extern "C" {

uint64_t wc_q4_bytes(uint64_t rows, uint64_t cols, uint32_t group, uint32_t flags) {
    if (!q4_shape_ok(rows, cols, group) || (flags & ~kStreamFlags) != 0) return 0;
    return wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags).total;
}

int wc_q4_quantize(const void* d_w, uint64_t ld, uint64_t rows, uint64_t cols, uint32_t group,
                   uint32_t flags, void* d_out, uint64_t out_capacity, void* stream) {
    if (!q4_shape_ok(rows, cols, group) || (flags & ~kStreamFlags) != 0 || d_out == nullptr ||
        !aligned(d_out, 16) || (rows > 0 && (d_w == nullptr || !aligned(d_w, 2) || ld < cols)))
        return WC_ERR_INVALID_ARG;
    const wc::Q4Layout L = wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags);
    if (out_capacity < L.total) return WC_ERR_BUFFER_TOO_SMALL;
    return result(wc::launch_q4_quantize(d_w, ld, L, static_cast<uint8_t*>(d_out),
                                         static_cast<cudaStream_t>(stream)));
}

int wc_q4_pack(const uint8_t* d_codes, const void* d_scales, const uint8_t* d_zeros, uint64_t rows,
               uint64_t cols, uint32_t group, uint32_t flags, void* d_out, uint64_t out_capacity,
               void* stream) {
    if (!q4_shape_ok(rows, cols, group) || (flags & ~kStreamFlags) != 0 || d_out == nullptr ||
        !aligned(d_out, 16) || (rows > 0 && (d_codes == nullptr || d_scales == nullptr ||
                                             !aligned(d_scales, 2))) ||
        (rows > 0 && (d_zeros != nullptr) != ((flags & WC_Q4_ZEROS) != 0)))
        return WC_ERR_INVALID_ARG;
    const wc::Q4Layout L = wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags);
    if (out_capacity < L.total) return WC_ERR_BUFFER_TOO_SMALL;
    return result(wc::launch_q4_pack(d_codes, d_scales, d_zeros, L, static_cast<uint8_t*>(d_out),
                                     static_cast<cudaStream_t>(stream)));
}

int wc_q4_dequantize(const void* d_stream, uint64_t stream_bytes, uint64_t rows, uint64_t cols,
                     uint32_t group, uint32_t flags, void* d_out, uint64_t ld, uint32_t dtype,
                     int32_t* d_status, void* stream) {
    if ((flags & ~kStreamFlags) != 0 || dtype > WC_DTYPE_FP32) return WC_ERR_INVALID_ARG;
    const int rc = check_stream(d_stream, stream_bytes, rows, cols, group, flags);
    if (rc != WC_OK) return rc;
    if (rows > 0 && (d_out == nullptr || !aligned(d_out, dtype_size(dtype)) || ld < cols))
        return WC_ERR_INVALID_ARG;
    const wc::Q4Layout L = wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags);
    return result(wc::launch_q4_dequantize(static_cast<const uint8_t*>(d_stream), L, d_out, ld,
                                           dtype, d_status, static_cast<cudaStream_t>(stream)));
}

static int q4_product(const void* d_streams, uint64_t stride, uint32_t experts, uint64_t rows,
                      uint64_t cols, uint32_t group, uint32_t flags, const void* d_x, uint64_t ldx,
                      uint64_t tokens, const int32_t* d_offsets, void* d_y, uint64_t ldy,
                      int32_t* d_status, void* stream) {
    if (tokens > WC_Q4_MAX_TOKENS) return WC_ERR_INVALID_ARG;
    if (rows > 0 && tokens > 0) {
        if (d_x == nullptr || d_y == nullptr || !aligned(d_x, 2) ||
            !aligned(d_y, flags & WC_Q4_Y_16BIT ? 2 : 4) || ldx < cols || ldy < rows)
            return WC_ERR_INVALID_ARG;
    }
    wc::Q4GemmArgs a;
    a.stream = static_cast<const uint8_t*>(d_streams);
    a.stride = stride;
    a.experts = experts;
    a.x = d_x;
    a.ldx = ldx;
    a.y = d_y;
    a.ldy = ldy;
    a.tokens = uint32_t(tokens);
    a.offsets = d_offsets;
    a.flags = flags;
    a.status = d_status;
    const wc::Q4Layout L = wc::q4_layout(uint32_t(rows), uint32_t(cols), group, flags);
    const bool few = d_offsets == nullptr ? tokens <= kFewRows
                                          : tokens <= uint64_t(experts) * kFewRowsExperts;
    const auto launch = few ? wc::launch_q4_gemv : wc::launch_q4_gemm;
    return result(launch(a, L, static_cast<cudaStream_t>(stream)));
}

int wc_q4_gemm(const void* d_stream, uint64_t stream_bytes, uint64_t rows, uint64_t cols,
               uint32_t group, uint32_t flags, const void* d_x, uint64_t ldx, uint64_t tokens,
               void* d_y, uint64_t ldy, int32_t* d_status, void* stream) {
    if ((flags & ~kAllFlags) != 0) return WC_ERR_INVALID_ARG;
    const int rc = check_stream(d_stream, stream_bytes, rows, cols, group, flags);
    if (rc != WC_OK) return rc;
    return q4_product(d_stream, 0, 1, rows, cols, group, flags, d_x, ldx, tokens, nullptr, d_y, ldy,
                      d_status, stream);
}

int wc_q4_gemm_experts(const void* d_streams, uint64_t stream_stride, uint32_t experts,
                       uint64_t rows, uint64_t cols, uint32_t group, uint32_t flags,
                       const void* d_x, uint64_t ldx, uint64_t tokens, const int32_t* d_offsets,
                       void* d_y, uint64_t ldy, int32_t* d_status, void* stream) {
    if ((flags & ~kAllFlags) != 0 || experts < 1 || experts > WC_MOE_MAX_EXPERTS ||
        d_offsets == nullptr || !aligned(d_offsets, 4) || stream_stride % 16 != 0)
        return WC_ERR_INVALID_ARG;
    const int rc = check_stream(d_streams, stream_stride, rows, cols, group, flags);
    if (rc != WC_OK) return rc;
    return q4_product(d_streams, stream_stride, experts, rows, cols, group, flags, d_x, ldx, tokens,
                      d_offsets, d_y, ldy, d_status, stream);
}

int wc_moe_sort(const int32_t* d_ids, uint64_t slots, uint32_t experts, int32_t* d_offsets,
                int32_t* d_order, int32_t* d_inverse, void* stream) {
    if (experts < 1 || experts > WC_MOE_MAX_EXPERTS || slots > WC_MOE_MAX_SLOTS ||
        d_offsets == nullptr || !aligned(d_offsets, 4) || !aligned(d_order, 4) ||
        (slots > 0 && (d_ids == nullptr || d_inverse == nullptr)) || !aligned(d_ids, 4) ||
        !aligned(d_inverse, 4))
        return WC_ERR_INVALID_ARG;
    return result(wc::launch_moe_sort(d_ids, uint32_t(slots), experts, d_offsets, d_order, d_inverse,
                                      static_cast<cudaStream_t>(stream)));
}

// The arguments that the three row operators share.
static int moe_args(uint64_t tokens, uint64_t top, uint64_t cols, uint32_t dtype,
                    const int32_t* d_inverse, uint64_t rows, wc::MoeArgs* a) {
    if (dtype > WC_DTYPE_FP32 || cols > WC_MOE_MAX_COLS || tokens > WC_MOE_MAX_SLOTS ||
        top > WC_MOE_MAX_SLOTS || tokens * top > WC_MOE_MAX_SLOTS || rows > WC_MOE_MAX_SLOTS ||
        (tokens * top > 0 && d_inverse == nullptr) || !aligned(d_inverse, 4))
        return WC_ERR_INVALID_ARG;
    a->tokens = tokens;
    a->top = uint32_t(top);
    a->cols = cols;
    a->dtype = dtype;
    a->inverse = d_inverse;
    a->rows = rows;
    return WC_OK;
}

// A matrix of `n` rows: given, aligned to its elements, its rows apart.
static bool moe_matrix(const void* p, uint64_t n, uint64_t cols, uint64_t ld, uint32_t dtype) {
    return n == 0 || cols == 0 || (p != nullptr && aligned(p, dtype_size(dtype)) && ld >= cols);
}

int wc_moe_gather(const void* d_x, uint64_t ldx, uint64_t tokens, uint64_t top, uint64_t cols,
                  uint32_t dtype, const int32_t* d_inverse, void* d_rows, uint64_t ldr,
                  uint64_t rows, void* stream) {
    wc::MoeArgs a;
    const int rc = moe_args(tokens, top, cols, dtype, d_inverse, rows, &a);
    if (rc != WC_OK) return rc;
    if (!moe_matrix(d_x, tokens, cols, ldx, dtype) || !moe_matrix(d_rows, rows, cols, ldr, dtype))
        return WC_ERR_INVALID_ARG;
    return result(
        wc::launch_moe_gather(a, d_x, ldx, d_rows, ldr, static_cast<cudaStream_t>(stream)));
}

int wc_moe_combine(const void* d_rows, uint64_t ldr, uint64_t rows, uint64_t tokens, uint64_t top,
                   uint64_t cols, uint32_t dtype, const int32_t* d_inverse, const float* d_weights,
                   void* d_out, uint64_t ldo, void* stream) {
    wc::MoeArgs a;
    const int rc = moe_args(tokens, top, cols, dtype, d_inverse, rows, &a);
    if (rc != WC_OK) return rc;
    if (!moe_matrix(d_rows, rows, cols, ldr, dtype) || !moe_matrix(d_out, tokens, cols, ldo, dtype) ||
        !aligned(d_weights, 4))
        return WC_ERR_INVALID_ARG;
    return result(wc::launch_moe_combine(a, d_rows, ldr, d_weights, d_out, ldo,
                                         static_cast<cudaStream_t>(stream)));
}

int wc_moe_combine_backward(const void* d_dout, uint64_t ldd, const void* d_rows, uint64_t ldr,
                            uint64_t rows, uint64_t tokens, uint64_t top, uint64_t cols,
                            uint32_t dtype, const int32_t* d_inverse, const float* d_weights,
                            void* d_drows, uint64_t lddr, float* d_dweights, void* stream) {
    wc::MoeArgs a;
    const int rc = moe_args(tokens, top, cols, dtype, d_inverse, rows, &a);
    if (rc != WC_OK) return rc;
    if (!moe_matrix(d_dout, tokens, cols, ldd, dtype) || !moe_matrix(d_rows, rows, cols, ldr, dtype) ||
        !moe_matrix(d_drows, rows, cols, lddr, dtype) || !aligned(d_weights, 4) ||
        !aligned(d_dweights, 4))
        return WC_ERR_INVALID_ARG;
    return result(wc::launch_moe_combine_backward(a, d_dout, ldd, d_rows, ldr, d_weights, d_drows,
                                                  lddr, d_dweights,
                                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
