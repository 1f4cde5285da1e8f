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
    uint32_t split;   // thread blocks of a cluster, which share the slices
    bool vec;         // rows of x are 16-byte aligned
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
__device__ __forceinline__ uint4 load_x8(const uint16_t* row, uint32_t c, uint32_t cols, bool vec) {
    if (vec && c + 8 <= cols) return __ldg(reinterpret_cast<const uint4*>(row + c));
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)
        if (c + k < cols) v[k >> 1] |= uint32_t(__ldg(row + c + k)) << (16 * (k & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One warp's slice: RT 16-row records against NT x 8 rows of x. PER: groups of
// the slice's 128 columns.
template <bool HALF, int RT, int NT, int PER>
__device__ __forceinline__ void slice_mma(const uint4 (&c0)[RT], const uint4 (&c1)[RT],
                                          const uint16_t (&s0)[RT][PER], const uint16_t (&s1)[RT][PER],
                                          const uint32_t (&z0)[RT][PER], const uint32_t (&z1)[RT][PER],
                                          const uint4 (&xv)[NT][4], uint32_t half_scales,
                                          const Q4Masks& mk,
                                          float (&acc)[RT][NT][4]) {
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
                const uint32_t w0 = word_of(c0[r], i), w1 = word_of(c1[r], i);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t a0 = q4_pair<HALF>(w0, 2 * m, z0[r][g], mk);
                    const uint32_t a1 = q4_pair<HALF>(w1, 2 * m, z1[r][g], mk);
                    const uint32_t a2 = q4_pair<HALF>(w0, 2 * m + 1, z0[r][g], mk);
                    const uint32_t a3 = q4_pair<HALF>(w1, 2 * m + 1, z1[r][g], mk);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<HALF>(part[r][n], a0, a1, a2, a3, word_of(xv[n][i], 2 * m),
                                       word_of(xv[n][i], 2 * m + 1));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const float f0 = q4_scale(s0[r][g], half_scales), f1 = q4_scale(s1[r][g], half_scales);
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

template <bool HALF, int RT, int NT, int PER>
__global__ void __launch_bounds__(kGvThreads) q4_gemv_kernel(const __grid_constant__ GvParams P) {
    const Q4Layout& L = P.L;
    const Q4GemmArgs& A = P.a;
    __shared__ float sums[kWarps][RT * NT * 4][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t = lane & 3;
    const uint32_t part = blockIdx.x % P.split;         // rank in the cluster
    const uint32_t b0 = blockIdx.x / P.split * RT;      // first 16-row block
    const uint32_t e = blockIdx.y;
    uint32_t lo = 0, hi = A.tokens;
    if (A.offsets != nullptr) {
        lo = uint32_t(min(max(A.offsets[e], 0), int(A.tokens)));
        hi = uint32_t(min(max(A.offsets[e + 1], int(lo)), int(A.tokens)));
    }
    const uint8_t* stream = A.stream + e * A.stride;
    if (blockIdx.x == 0 && threadIdx.x == 0 && hi > lo) q4_check_header(stream, L, A.status);
    const uint32_t h = min(8u, L.blocks16 - (b0 & ~7u));
    const Q4Masks mk = Q4Masks::make<HALF>();
    const uint32_t nrec = min(uint32_t(RT), L.blocks16 - b0);
    for (uint32_t t0 = lo; t0 < hi; t0 += 8 * NT) {
        float acc[RT][NT][4] = {};
        for (uint32_t s = part * kWarps + warp; s < L.slices; s += P.split * kWarps) {
            const uint8_t* rec = stream + q4_record(L, b0, s);
            uint4 c0[RT], c1[RT], xv[NT][4];
            uint16_t s0[RT][PER], s1[RT][PER];
            uint32_t z0[RT][PER], z1[RT][PER];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint8_t* p = rec + (uint32_t(r) < nrec ? r : 0) * L.rec;
                c0[r] = ld_stream_v4(p + t * 256 + g * 16);
                c1[r] = ld_stream_v4(p + t * 256 + g * 16 + 128);
                const uint16_t* sp = reinterpret_cast<const uint16_t*>(p + kQ4Codes);
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    s0[r][k] = __ldg(sp + k * 16 + g);
                    s1[r][k] = __ldg(sp + k * 16 + g + 8);
                    const uint8_t* zp = p + kQ4Codes + 32 * PER + k * 16 + g;
                    z0[r][k] = q4_zero_pair<HALF>(L.zeros ? __ldg(zp) : 8u);
                    z1[r][k] = q4_zero_pair<HALF>(L.zeros ? __ldg(zp + 8) : 8u);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t tok = t0 + 8 * n + g;
                const uint16_t* row = static_cast<const uint16_t*>(A.x) + uint64_t(tok) * A.ldx;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    xv[n][i] = tok < hi ? load_x8(row, s * kQ4Cols + 32 * i + 8 * t, L.cols, P.vec)
                                        : make_uint4(0, 0, 0, 0);
            }
            slice_mma<HALF, RT, NT, PER>(c0, c1, s0, s1, z0, z1, xv, L.half_scales, mk, acc);
        }
        // partial sums of the block's warps, then of the cluster's blocks, in a fixed order
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) sums[warp][(r * NT + n) * 4 + k][lane] = acc[r][n][k];
        __syncthreads();
        constexpr int kVals = RT * NT * 4 * 32;
        for (uint32_t v = threadIdx.x; v < kVals; v += kGvThreads) {
            float sum = 0.f;
            for (int w = 0; w < kWarps; ++w) sum += (&sums[w][0][0])[v];
            (&sums[0][0][0])[v] = sum;
        }
        if (P.split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
        if (part == 0) {
            for (uint32_t v = threadIdx.x; v < kVals; v += kGvThreads) {
                // consecutive threads take consecutive rows of one token
                const uint32_t row = v % (RT * 16), tok = v / (RT * 16);
                const uint32_t r = row >> 4, gg = row & 7u, up = (row >> 3) & 1u;
                const uint32_t n = tok >> 3, tt = (tok & 7u) >> 1, odd = tok & 1u;
                const uint32_t at = ((r * NT + n) * 4 + up * 2 + odd) * 32 + gg * 4 + tt;
                float sum = 0.f;
                if (P.split > 1) {
                    for (uint32_t q = 0; q < P.split; ++q)
                        sum += cg::this_cluster().map_shared_rank(&sums[0][0][0], q)[at];
                } else {
                    sum = (&sums[0][0][0])[at];
                }
                const uint32_t R = b0 * kQ4Rows + row, p = t0 + tok;
                if (R < L.rows && p < hi) {
                    if (A.flags & kQ4Y16) {
                        uint16_t* y = static_cast<uint16_t*>(A.y) + uint64_t(p) * A.ldy + R;
                        *y = HALF ? __half_as_ushort(__float2half_rn(sum))
                                  : __bfloat16_as_ushort(__float2bfloat16_rn(sum));
                    } else {
                        static_cast<float*>(A.y)[uint64_t(p) * A.ldy + R] = sum;
                    }
                }
            }
        }
        if (P.split > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
}

template <bool HALF, int RT, int NT, int PER>
cudaError_t gv_launch(const GvParams& P, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((P.L.blocks16 + RT - 1) / RT * P.split, P.a.experts);
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

}  // namespace

cudaError_t launch_q4_gemv(const Q4GemmArgs& a, const Q4Layout& L, cudaStream_t stream) {
    if (L.rows == 0 || a.tokens == 0) return cudaSuccess;
    GvParams P;
    P.a = a;
    P.L = L;
    P.vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ldx % 8 == 0;
    P.split = 1;
    return a.flags & kQ4XHalf ? gv_per<true, 2, 1>(P, stream) : gv_per<false, 2, 1>(P, stream);
}

}  // namespace wc
