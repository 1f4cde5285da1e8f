// wc_q4_core.cuh -- layout and unpacking of 4-bit streams with group scales
// (sm_100a), shared by the quantizer and the fused products.
//
// A weight is W[r][c] = s * (q - z): a 4-bit code q, and a 16-bit scale s and
// (optionally) a 4-bit zero point z for each row and group of 32, 64 or 128
// consecutive columns; z = 8 without zero points. The stream is a 128-byte
// container header and records of 16 rows x 128 columns; rows and columns are
// padded to whole records with codes that stand for zero (and scale 0 where a
// whole group is padding). A record:
//   1024 bytes of codes: 32-bit words [t 0..3][row 0..15][i 0..3]; word (t, i)
//     holds columns 32 i + 8 t + (0..7) of its row, element e in nibble
//     (e >> 1) + 4 (e & 1)
//   scales u16 [128 / group][16 rows]
//   with zero points: u8 [128 / group][16 rows], padded to 32 bytes
// ordered [128-row block][128-column slice][16-row block of the 128].
// Why this order: a 16-byte piece holds four words of one row that lie 32
// columns apart, so a lane that owns (row, t) has what the fragments of a
// 16 x 8 x 16 matrix instruction need for any of the group sizes, and a warp
// reads whole 128-byte lines; a lane that owns a row finds the row's pieces
// free of bank conflicts in shared memory; and a 128 x 128 tile is one
// contiguous piece. The nibble order makes (word >> 4 k) & 0x000F000F the pair
// of elements 2 k and 2 k + 1 in the two 16-bit halves.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "wc_internal.cuh"

namespace wc {

constexpr uint32_t kFlagQ4 = 8;         // header flags: a 4-bit stream,
constexpr uint32_t kFlagQ4Zeros = 16;   // with zero points,
constexpr uint32_t kFlagQ4Half = 32;    // scales in FP16 (else BF16)
constexpr uint32_t kQ4Rows = 16;        // rows of a record
constexpr uint32_t kQ4Cols = 128;       // columns of a record
constexpr uint32_t kQ4Codes = 1024;     // bytes of codes of a record

// caller's flags (the values of WC_Q4_*)
constexpr uint32_t kQ4Zeros = 1, kQ4ScalesHalf = 2, kQ4XHalf = 4, kQ4Y16 = 8;

struct Q4Layout {
    uint32_t rows, cols, group;
    uint32_t per;       // groups of a record's 128 columns: 1, 2 or 4
    uint32_t rec;       // bytes of a record
    uint32_t blocks16;  // 16-row blocks
    uint32_t slices;    // 128-column slices
    uint32_t zeros, half_scales;
    uint64_t total;     // stream bytes
};

__host__ __device__ inline bool q4_group_ok(uint32_t g) { return g == 32 || g == 64 || g == 128; }

__host__ __device__ inline Q4Layout q4_layout(uint32_t rows, uint32_t cols, uint32_t group,
                                              uint32_t flags) {
    Q4Layout L;
    L.rows = rows;
    L.cols = cols;
    L.group = group;
    L.per = kQ4Cols / group;
    L.zeros = flags & kQ4Zeros ? 1u : 0u;
    L.half_scales = flags & kQ4ScalesHalf ? 1u : 0u;
    L.rec = kQ4Codes + 32u * L.per + (L.zeros ? (16u * L.per + 31u) / 32u * 32u : 0u);
    L.blocks16 = uint32_t((uint64_t(rows) + kQ4Rows - 1) / kQ4Rows);
    L.slices = uint32_t((uint64_t(cols) + kQ4Cols - 1) / kQ4Cols);
    L.total = kHeaderBytes + uint64_t(L.blocks16) * L.slices * L.rec;
    return L;
}

// Byte offset of record (16-row block b, slice s); block b + 1 of the same 128
// rows follows directly.
__host__ __device__ inline uint64_t q4_record(const Q4Layout& L, uint32_t b, uint32_t s) {
    const uint32_t first = b & ~7u;
    const uint32_t h = L.blocks16 - first < 8u ? L.blocks16 - first : 8u;
    return kHeaderBytes + (uint64_t(first) * L.slices + uint64_t(s) * h + (b - first)) * L.rec;
}

// 64-bit word k (0..15) of the container header.
__host__ __device__ inline uint64_t q4_header_word(const Q4Layout& L, int k) {
    switch (k) {
        case 0: return kMagic | (uint64_t(kVersion) << 32) | (uint64_t(kHeaderBytes) << 48);
        case 1:
            return uint64_t(L.group) |
                   (uint64_t(kFlagQ4 | (L.zeros ? kFlagQ4Zeros : 0u) |
                             (L.half_scales ? kFlagQ4Half : 0u))
                    << 32);
        case 2: return uint64_t(L.rows) * L.cols;
        case 3: return uint64_t(L.rows) * ((uint64_t(L.cols) + L.group - 1) / L.group);
        case 4: return kHeaderBytes;
        case 8: return L.total - kHeaderBytes;
        case 9: return L.total;
        case 11: return uint64_t(L.rows) | (uint64_t(L.cols) << 32);
        default: return 0;
    }
}

// The container header against what the caller states (one thread).
__device__ inline void q4_check_header(const uint8_t* stream, const Q4Layout& L, int32_t* status) {
    bool bad = false;
    for (int k = 0; k < 16; ++k)
        bad |= reinterpret_cast<const uint64_t*>(stream)[k] != q4_header_word(L, k);
    if (bad) report(status, kStatusCorrupt);
}

__device__ __forceinline__ float q4_scale(uint16_t bits, uint32_t half_scales) {
    return half_scales ? __half2float(__ushort_as_half(bits))
                       : __uint_as_float(uint32_t(bits) << 16);
}

// Two 16-bit floats 2^m + q with the code q in the lowest mantissa bits:
// 128 + q in BF16, 1024 + q in FP16. Subtracting the pair of 2^m + z gives
// q - z exactly: at most 4 significant bits.
template <bool HALF>
__host__ __device__ constexpr uint32_t q4_magic() {
    return HALF ? 0x64006400u : 0x43004300u;
}

template <bool HALF>
__device__ __forceinline__ uint32_t q4_zero_pair(uint32_t z) {
    return q4_magic<HALF>() | (z & 15u) * 0x00010001u;
}

// The masks of the unpacking, kept in registers: an instruction takes one
// immediate, so with both as immediates (x & mask) | magic would be two.
struct Q4Masks {
    uint32_t mask, magic;
    template <bool HALF>
    static __device__ __forceinline__ Q4Masks make() {
        Q4Masks m;
        asm volatile("mov.u32 %0, %1;" : "=r"(m.mask) : "n"(0x000F000F));
        asm volatile("mov.u32 %0, %1;" : "=r"(m.magic) : "n"(q4_magic<HALF>()));
        return m;
    }
};

// The pair of elements 2 k and 2 k + 1 of a word as q - z.
template <bool HALF>
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int k, uint32_t zero_pair,
                                            const Q4Masks& m) {
    uint32_t v, d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"  // (a & b) | c
        : "=r"(v)
        : "r"(word >> (4 * k)), "r"(m.mask), "r"(m.magic));
    if (HALF)
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(zero_pair));
    else
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(zero_pair));
    return d;
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
struct Q4GemmArgs {
    const uint8_t* stream;   // first matrix; matrix e at stream + e * stride
    uint64_t stride;
    uint32_t experts;        // matrices
    const void* x;           // rows of activations, ldx elements apart
    uint64_t ldx;
    void* y;                 // rows of results, ldy elements apart
    uint64_t ldy;
    uint32_t tokens;         // rows of x and y
    const int32_t* offsets;  // experts + 1 first rows (nullptr: one matrix, all rows)
    uint32_t flags;
    int32_t* status;
};

// Result y[row of x][row of W], rounded once if it is to be 16 bits.
template <bool HALF>
__device__ __forceinline__ void q4_store(const Q4GemmArgs& a, uint64_t tok, uint32_t row, float v) {
    if (a.flags & kQ4Y16)
        static_cast<uint16_t*>(a.y)[tok * a.ldy + row] =
            HALF ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        static_cast<float*>(a.y)[tok * a.ldy + row] = v;
}

cudaError_t launch_q4_quantize(const void* w, uint64_t ld, const Q4Layout& L, uint8_t* out,
                               cudaStream_t stream);
cudaError_t launch_q4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros,
                           const Q4Layout& L, uint8_t* out, cudaStream_t stream);
cudaError_t launch_q4_dequantize(const uint8_t* in, const Q4Layout& L, void* out, uint64_t ld,
                                 uint32_t dtype, int32_t* status, cudaStream_t stream);
// Products with few rows of x a matrix (wc_q4_gemv.cu) and with many (wc_q4_gemm.cu).
cudaError_t launch_q4_gemv(const Q4GemmArgs& a, const Q4Layout& L, cudaStream_t stream);
cudaError_t launch_q4_gemm(const Q4GemmArgs& a, const Q4Layout& L, cudaStream_t stream);

struct MoeArgs {
    uint64_t tokens;
    uint32_t top;
    uint64_t cols;
    uint32_t dtype;          // 0 BF16, 1 FP16, 2 FP32
    const int32_t* inverse;  // tokens x top: row of each slot, or outside 0..rows-1: none
    uint64_t rows;           // rows of the sorted matrices
};

cudaError_t launch_moe_sort(const int32_t* ids, uint32_t slots, uint32_t experts, int32_t* offsets,
                            int32_t* order, int32_t* inverse, cudaStream_t stream);
cudaError_t launch_moe_gather(const MoeArgs& a, const void* x, uint64_t ldx, void* out,
                              uint64_t ldo, cudaStream_t stream);
cudaError_t launch_moe_combine(const MoeArgs& a, const void* y, uint64_t ldy, const float* weights,
                               void* out, uint64_t ldo, cudaStream_t stream);
cudaError_t launch_moe_combine_backward(const MoeArgs& a, const void* dout, uint64_t ldd,
                                        const void* y, uint64_t ldy, const float* weights,
                                        void* dy, uint64_t lddy, float* dweights,
                                        cudaStream_t stream);

}  // namespace wc
