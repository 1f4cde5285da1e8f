// wc_q4_gemv.cu -- products of 4-bit weights with a few rows of activations.
//
//   y[p][r] = sum_g s[r][g] * sum_{c in g} (q[r][c] - z[r][g]) * x[p][c]
//
// for the rows p of each matrix's range, W held only as its 4-bit stream. The
// codes become exact 16-bit integers q - z in registers and go through
// 16 x 8 x 16 matrix instructions with FP32 accumulators, weights as the
// 16-row operand and up to 8 rows of x as the 8 columns; each group's sum is
// then scaled once into a second FP32 accumulator. So no scaled weight is ever
// rounded, and a weight costs about 1.4 instructions. At these row counts the
// time is the stream's bytes.
#include <cooperative_groups.h>

#include <mutex>

#include "wc_q4_core.cuh"

namespace wc {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kGvThreads = 32 * kWarps;

struct GvParams {
    Q4GemmArgs a;
    Q4Layout L;
    uint32_t wk;       // warps that share a row group's slices (a power of two up to 8)
    uint32_t split;    // thread blocks of a cluster that share them, too
    uint32_t x_bytes;  // bytes (2 to 16) that divide the address of every row of x
};

template <bool HALF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight activations of a row from column c, zeros past the end.
__device__ __forceinline__ uint4 load_x8(const uint16_t* row, uint32_t c, uint32_t cols,
                                         uint32_t x_bytes) {
    if (x_bytes >= 4 && c + 8 <= cols) {
        if (x_bytes == 16) return __ldg(reinterpret_cast<const uint4*>(row + c));
        if (x_bytes == 8) {
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + c));
            const uint2 b = __ldg(reinterpret_cast<const uint2*>(row + c + 4));
            return make_uint4(a.x, a.y, b.x, b.y);
        }
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row + c);
        return make_uint4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
    }
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (c + k < cols) v[k >> 1] |= uint32_t(__ldg(row + c + k)) << (16 * (k & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// What a warp reads of one slice: RT 16-row records (each lane 16 bytes of codes
// of the rows g and g + 8, their scales and zero points) and NT x 8 rows of x.
template <int RT, int NT, int PER>
struct Slice {
    uint4 c0[RT], c1[RT], x[NT][4];
    uint16_t s0[RT][PER], s1[RT][PER];
    uint8_t z0[RT][PER], z1[RT][PER];
};

template <int RT, int NT, int PER>
__device__ __forceinline__ void load_slice(Slice<RT, NT, PER>& v, const GvParams& P,
                                           const uint8_t* stream, uint32_t b0, uint32_t s,
                                           uint32_t nrec, uint32_t t0, uint32_t hi, uint32_t g,
                                           uint32_t t) {
    const Q4Layout& L = P.L;
    const uint8_t* rec = stream + q4_record(L, b0, s);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const uint8_t* p = rec + (uint32_t(r) < nrec ? r : 0) * L.rec;
        v.c0[r] = ld_stream_v4(p + t * 256 + g * 16);
        v.c1[r] = ld_stream_v4(p + t * 256 + g * 16 + 128);
        const uint16_t* sp = reinterpret_cast<const uint16_t*>(p + kQ4Codes);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            v.s0[r][k] = __ldg(sp + k * 16 + g);
            v.s1[r][k] = __ldg(sp + k * 16 + g + 8);
            const uint8_t* zp = p + kQ4Codes + 32 * PER + k * 16 + g;
            v.z0[r][k] = L.zeros ? __ldg(zp) : 8u;
            v.z1[r][k] = L.zeros ? __ldg(zp + 8) : 8u;
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint32_t tok = t0 + 8 * n + g;
        const uint16_t* row = static_cast<const uint16_t*>(P.a.x) + uint64_t(tok) * P.a.ldx;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v.x[n][i] = tok < hi ? load_x8(row, s * kQ4Cols + 32 * i + 8 * t, L.cols, P.x_bytes)
                                 : make_uint4(0, 0, 0, 0);
    }
}

template <bool HALF, int RT, int NT, int PER>
__device__ __forceinline__ void slice_mma(const Slice<RT, NT, PER>& v, uint32_t half_scales,
                                          const Q4Masks& mk, float (&acc)[RT][NT][4]) {
#pragma unroll
    for (int g = 0; g < PER; ++g) {
        float part[RT][NT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) part[r][n][k] = 0.f;
#pragma unroll
        for (int i = g * (4 / PER); i < (g + 1) * (4 / PER); ++i) {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t w0 = word_of(v.c0[r], i), w1 = word_of(v.c1[r], i);
                const uint32_t z0 = q4_zero_pair<HALF>(v.z0[r][g]);
                const uint32_t z1 = q4_zero_pair<HALF>(v.z1[r][g]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t a0 = q4_pair<HALF>(w0, 2 * m, z0, mk);
                    const uint32_t a1 = q4_pair<HALF>(w1, 2 * m, z1, mk);
                    const uint32_t a2 = q4_pair<HALF>(w0, 2 * m + 1, z0, mk);
                    const uint32_t a3 = q4_pair<HALF>(w1, 2 * m + 1, z1, mk);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<HALF>(part[r][n], a0, a1, a2, a3, word_of(v.x[n][i], 2 * m),
                                       word_of(v.x[n][i], 2 * m + 1));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float f0 = q4_scale(v.s0[r][g], half_scales), f1 = q4_scale(v.s1[r][g], half_scales);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[r][n][0] = fmaf(f0, part[r][n][0], acc[r][n][0]);
                acc[r][n][1] = fmaf(f0, part[r][n][1], acc[r][n][1]);
                acc[r][n][2] = fmaf(f1, part[r][n][2], acc[r][n][2]);
                acc[r][n][3] = fmaf(f1, part[r][n][3], acc[r][n][3]);
            }
        }
    }
}

// A block's 8 warps are 8 / wk row groups of RT records each, times wk warps
// that take the row group's slices in turns (the blocks of a cluster, too). The
// next slice is on its way while one is multiplied.
template <bool HALF, int RT, int NT, int PER>
__global__ void __launch_bounds__(kGvThreads, 2) q4_gemv_kernel(const __grid_constant__ GvParams P) {
    const Q4Layout& L = P.L;
    const Q4GemmArgs& A = P.a;
    constexpr int kVals = RT * NT * 4 * 32;  // results of a row group, padding included
    __shared__ float sums[kWarps][kVals];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t = lane & 3;
    const uint32_t part = blockIdx.x % P.split;  // rank in the cluster
    const uint32_t wk = warp & (P.wk - 1u), wr = warp / P.wk, groups = kWarps / P.wk;
    const uint32_t first = blockIdx.x / P.split * groups * RT;  // the block's first 16-row block
    const uint32_t b0 = first + wr * RT;
    const uint32_t e = blockIdx.y;
    uint32_t lo = 0, hi = A.tokens;
    if (A.offsets != nullptr) {
        lo = uint32_t(min(max(A.offsets[e], 0), int(A.tokens)));
        hi = uint32_t(min(max(A.offsets[e + 1], int(lo)), int(A.tokens)));
    }
    if (hi == lo) return;  // the same for all blocks of a cluster
    const uint8_t* stream = A.stream + e * A.stride;
    const uint32_t nrec = b0 < L.blocks16 ? min(uint32_t(RT), L.blocks16 - b0) : 0u;
    const Q4Masks mk = Q4Masks::make<HALF>();
    const uint32_t step = P.split * P.wk;
    for (uint32_t t0 = lo; t0 < hi; t0 += 8 * NT) {
        float acc[RT][NT][4] = {};
        if (nrec > 0) {
            Slice<RT, NT, PER> v0, v1;
            uint32_t s = part * P.wk + wk;
            if (s < L.slices) load_slice(v0, P, stream, b0, s, nrec, t0, hi, g, t);
            while (s < L.slices) {
                s += step;
                if (s < L.slices) load_slice(v1, P, stream, b0, s, nrec, t0, hi, g, t);
                slice_mma<HALF, RT, NT, PER>(v0, L.half_scales, mk, acc);
                if (s >= L.slices) break;
                s += step;
                if (s < L.slices) load_slice(v0, P, stream, b0, s, nrec, t0, hi, g, t);
                slice_mma<HALF, RT, NT, PER>(v1, L.half_scales, mk, acc);
            }
        }
        // partial sums of a row group's warps, then of the cluster's blocks, in a fixed order
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sums[warp][((r * NT + n) * 4 + k) * 32 + lane] = acc[r][n][k];
        if (P.split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        if (part == 0) {
            for (uint32_t v = threadIdx.x; v < groups * kVals; v += kGvThreads) {
                // consecutive threads take consecutive rows of one token
                const uint32_t row = v % (RT * 16), gr = v / (RT * 16) % groups;
                const uint32_t tok = v / (RT * 16) / groups;
                const uint32_t r = row >> 4, gg = row & 7u, up = (row >> 3) & 1u;
                const uint32_t n = tok >> 3, tt = (tok & 7u) >> 1, odd = tok & 1u;
                const uint32_t at = ((r * NT + n) * 4 + up * 2 + odd) * 32 + gg * 4 + tt;
                const uint32_t R = (first + gr * RT) * kQ4Rows + row, p = t0 + tok;
                if (R >= L.rows || p >= hi) continue;
                float sum = 0.f;
                for (uint32_t q = 0; q < P.split; ++q) {
                    const float* from =
                        P.split > 1 ? cg::this_cluster().map_shared_rank(&sums[0][0], q) : &sums[0][0];
                    for (uint32_t w = 0; w < P.wk; ++w) sum += from[(gr * P.wk + w) * kVals + at];
                }
                if (A.flags & kQ4Y16) {
                    uint16_t* y = static_cast<uint16_t*>(A.y) + uint64_t(p) * A.ldy + R;
                    *y = HALF ? __half_as_ushort(__float2half_rn(sum))
                              : __bfloat16_as_ushort(__float2bfloat16_rn(sum));
                } else {
                    static_cast<float*>(A.y)[uint64_t(p) * A.ldy + R] = sum;
                }
            }
        }
        if (P.split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) q4_check_header(stream, L, A.status);
}

template <bool HALF, int RT, int NT, int PER>
cudaError_t gv_launch(const GvParams& P, cudaStream_t stream) {
    const uint32_t rows = kWarps / P.wk * RT;  // records of a block
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((P.L.blocks16 + rows - 1) / rows * P.split, P.a.experts);
    cfg.blockDim = dim3(kGvThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, q4_gemv_kernel<HALF, RT, NT, PER>, P);
}

template <bool HALF, int RT, int NT>
cudaError_t gv_per(const GvParams& P, cudaStream_t stream) {
    return P.L.per == 1   ? gv_launch<HALF, RT, NT, 1>(P, stream)
           : P.L.per == 2 ? gv_launch<HALF, RT, NT, 2>(P, stream)
                          : gv_launch<HALF, RT, NT, 4>(P, stream);
}

template <bool HALF>
cudaError_t gv_tiles(const GvParams& P, int rt, int nt, cudaStream_t stream) {
    if (rt == 1) return nt == 1 ? gv_per<HALF, 1, 1>(P, stream) : gv_per<HALF, 1, 2>(P, stream);
    return nt == 1 ? gv_per<HALF, 2, 1>(P, stream) : gv_per<HALF, 2, 2>(P, stream);
}

}  // namespace

cudaError_t launch_q4_gemv(const Q4GemmArgs& a, const Q4Layout& L, cudaStream_t stream) {
    if (L.rows == 0 || a.tokens == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    GvParams P;
    P.a = a;
    P.L = L;
    const uint64_t al = reinterpret_cast<uintptr_t>(a.x) | (a.ldx * 2);
    P.x_bytes = al % 16 == 0 ? 16u : al % 8 == 0 ? 8u : al % 4 == 0 ? 4u : 2u;
    // Matrices that can have rows, and rows of x a matrix has on average.
    const uint32_t used = a.offsets == nullptr ? 1u : a.tokens < a.experts ? a.tokens : a.experts;
    const uint32_t rows = (a.tokens + used - 1) / used;
    const int nt = rows > 8 ? 2 : 1;
    // Enough blocks to fill the machine first, then long runs of slices for each
    // warp and two records at a time (x is read once for both).
    const uint64_t want = 2ull * uint32_t(sms);
    auto blocks = [&](uint32_t rt, uint32_t wk) {
        const uint32_t per = kWarps / wk * rt;
        return uint64_t(used) * ((L.blocks16 + per - 1) / per);
    };
    int rt = 2;
    P.wk = 1;
    while (P.wk < 8 && (L.slices / P.wk > 4 || blocks(2, P.wk) < want) && P.wk * 2 <= L.slices)
        P.wk *= 2;
    if (blocks(2, P.wk) < want) rt = 1;
    P.split = 1;
    while (P.split < 8 && blocks(uint32_t(rt), P.wk) * P.split * 2 <= want &&
           L.slices / (P.wk * P.split) >= 4)
        P.split *= 2;
    return a.flags & kQ4XHalf ? gv_tiles<true>(P, rt, nt, stream)
                              : gv_tiles<false>(P, rt, nt, stream);
}

}  // namespace wc
