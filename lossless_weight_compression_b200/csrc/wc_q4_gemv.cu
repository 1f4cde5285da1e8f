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
// time is the stream's bytes and how soon they are on their way: a thread block
// owns 128 weight rows (the blocks of a cluster share their slices of 128
// columns), and a producer warp keeps up to eight slices' records in flight,
// each one contiguous bulk copy, beside the slice's activations. Eight warps
// take one 16-row record each, so that the only sum across warps is the
// cluster's, over its blocks in a fixed order.
//
// Measured (GPU time, groups of 128, BF16, weights from HBM; beside it the time of
// the bytes at the copy's rate): 1 row of x through 4096 x 4096 7.0 us (1.3), 6.3
// from L2; through 4096 x 14336 12.8 us (4.7); 8 rows through 14336 x 4096 15.4 us
// (4.7), 16 rows 19.4 us; 48 rows over 64 experts of 2048 x 1024 16.9 us (8.3).
// From L2 instead they take 2 to 8 % less: bound by the warps' chains of unpacking
// and multiplying (issue 0.31 to 0.50 a cycle) and by each block's start, first
// loads and tail, which come once for every 35 to 135 KB of the stream.
// Loads straight into registers, with a row's slices spread over a block's warps,
// were 10 % faster for one row of x through 4096 x 4096, 10 to 60 % slower for
// experts and for 16 rows. Two sums a group instead of one, for shorter chains of
// matrix instructions: no gain, 15 % slower at 16 rows (registers).
#include <cooperative_groups.h>
#include <stddef.h>

#include <mutex>

#include "wc_q4_core.cuh"
#include "wc_ring.cuh"

namespace wc {
namespace {

namespace cg = cooperative_groups;

constexpr int kGvWarps = 8;                         // one record each
constexpr int kGvThreads = 32 * (kGvWarps + 1);     // and the producer
constexpr uint32_t kGvMaxStages = 8;

struct GvParams {
    Q4GemmArgs a;
    Q4Layout L;
    uint32_t split;    // thread blocks of a cluster, which share the slices
    uint32_t x_bytes;  // bytes (2 to 16) that divide the address of every row of x
    uint32_t pitch;    // bytes of a stage's records
};

struct GvCtl {
    unsigned long long full[kGvMaxStages], empty[kGvMaxStages];
    int abort;
};

// NT x 8 rows of x; a stage's activations are 256 bytes a row.
template <int NT>
struct GvShape {
    static constexpr uint32_t stages = NT == 1 ? 8 : 7;  // two blocks fit a multiprocessor
    static constexpr uint32_t x_bytes = NT * 8 * 256;
    static constexpr uint32_t vals = NT * 4 * 32;        // results of a record
};

template <int NT>
__host__ __device__ inline uint32_t gv_smem(uint32_t pitch) {
    return GvShape<NT>::stages * (pitch + GvShape<NT>::x_bytes) + kGvWarps * GvShape<NT>::vals * 4 +
           uint32_t((sizeof(GvCtl) + 15) / 16 * 16);
}

__device__ __forceinline__ bool gv_poll(unsigned long long* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait of a whole warp for a phase, its control flow uniform; false if another
// warp gave up or the time limit passed.
__device__ __forceinline__ bool gv_wait(unsigned long long* bar, uint32_t parity, GvCtl& c,
                                        int32_t* status) {
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 128; ++k)
            if (__all_sync(0xFFFFFFFFu, gv_poll(bar, parity))) return true;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        const bool late = t - t0 > kWaitLimitNs;
        if (__any_sync(0xFFFFFFFFu, late || *const_cast<volatile int*>(&c.abort))) {
            if (late) report(status, kStatusTimeout);
            c.abort = 1;
            return false;
        }
    }
}

// Byte b of row n of a stage's activations: 16-byte pieces, those of odd rows
// swapped in fours, so that the eight lanes of two rows read all banks.
__device__ __forceinline__ uint32_t gv_x_at(uint32_t n, uint32_t b) {
    return n * 256u + (b ^ ((n & 1u) << 6));
}

// The slice's activations by V-byte copies (16, 8, 4: cp.async; 2: through
// registers), zeros past the last column. Rows past the range are not copied:
// whatever their columns of the product hold is not stored.
template <int V>
__device__ __forceinline__ void gv_copy_x(const GvParams& P, uint32_t dst, uint32_t t0, uint32_t ntok,
                                          uint32_t s, uint32_t lane) {
    constexpr uint32_t W = V == 2 ? 4 : V;
    constexpr uint32_t per_row = 256 / W;
    for (uint32_t k = lane; k < ntok * per_row; k += 32) {
        const uint32_t n = k / per_row, b = (k % per_row) * W;
        const uint32_t col = s * kQ4Cols + b / 2;
        const uint16_t* src =
            static_cast<const uint16_t*>(P.a.x) + uint64_t(t0 + n) * P.a.ldx + col;
        const uint32_t have = col < P.L.cols ? min(W, (P.L.cols - col) * 2) : 0u;
        const uint32_t at = dst + gv_x_at(n, b);
        if (V == 2) {
            const uint32_t v = (have >= 2 ? uint32_t(src[0]) : 0u) |
                               (have >= 4 ? uint32_t(src[1]) << 16 : 0u);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
        } else {
            const void* from = have ? static_cast<const void*>(src) : P.a.x;
            if (V == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from),
                             "r"(have)
                             : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(from),
                             "n"(V == 2 ? 4 : V == 16 ? 4 : V), "r"(have)
                             : "memory");
        }
    }
}

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

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ uint4 gv_lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a));
    return v;
}

// One record of a slice (at `rec` in shared memory) against NT x 8 rows of x.
template <bool HALF, int NT, int PER>
__device__ __forceinline__ void record_mma(uint32_t rec, uint32_t x, uint32_t zeros,
                                           uint32_t half_scales, uint32_t g, uint32_t t,
                                           const Q4Masks& mk, float (&acc)[NT][4]) {
    const uint4 c0 = gv_lds128(rec + t * 256 + g * 16);
    const uint4 c1 = gv_lds128(rec + t * 256 + g * 16 + 128);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        uint16_t b0, b1;
        const uint32_t sp = rec + kQ4Codes + (k * 16 + g) * 2;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b0) : "r"(sp));
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(b1) : "r"(sp + 16));
        uint32_t z0 = 8, z1 = 8;
        if (zeros) {
            const uint32_t zp = rec + kQ4Codes + 32 * PER + k * 16 + g;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z0) : "r"(zp));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(z1) : "r"(zp + 8));
        }
        const uint32_t p0 = q4_zero_pair<HALF>(z0), p1 = q4_zero_pair<HALF>(z1);
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[n][j] = 0.f;
#pragma unroll
        for (int i = k * (4 / PER); i < (k + 1) * (4 / PER); ++i) {
            const uint32_t w0 = word_of(c0, i), w1 = word_of(c1, i);
            uint4 xv[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xv[n] = gv_lds128(x + gv_x_at(8 * n + g, 64 * i + 16 * t));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t a0 = q4_pair<HALF>(w0, 2 * m, p0, mk);
                const uint32_t a1 = q4_pair<HALF>(w1, 2 * m, p1, mk);
                const uint32_t a2 = q4_pair<HALF>(w0, 2 * m + 1, p0, mk);
                const uint32_t a3 = q4_pair<HALF>(w1, 2 * m + 1, p1, mk);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816<HALF>(part[n], a0, a1, a2, a3, word_of(xv[n], 2 * m),
                                   word_of(xv[n], 2 * m + 1));
            }
        }
        const float f0 = q4_scale(b0, half_scales), f1 = q4_scale(b1, half_scales);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(f0, part[n][0], acc[n][0]);
            acc[n][1] = fmaf(f0, part[n][1], acc[n][1]);
            acc[n][2] = fmaf(f1, part[n][2], acc[n][2]);
            acc[n][3] = fmaf(f1, part[n][3], acc[n][3]);
        }
    }
}

template <bool HALF, int NT, int PER>
__global__ void __launch_bounds__(kGvThreads, 2) q4_gemv_kernel(const __grid_constant__ GvParams P) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    const Q4Layout& L = P.L;
    const Q4GemmArgs& A = P.a;
    using Shape = GvShape<NT>;
    uint8_t* w_ring = smem_raw;
    uint8_t* x_ring = w_ring + Shape::stages * P.pitch;
    float* sums = reinterpret_cast<float*>(x_ring + Shape::stages * Shape::x_bytes);
    GvCtl& c = *reinterpret_cast<GvCtl*>(sums + kGvWarps * Shape::vals);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const uint32_t g = lane >> 2, t = lane & 3;
    const uint32_t part = blockIdx.x % P.split;  // rank in the cluster
    const uint32_t b0 = blockIdx.x / P.split * 8;
    const uint32_t e = blockIdx.y;
    uint32_t lo = 0, hi = A.tokens;
    if (A.offsets != nullptr) {
        lo = uint32_t(min(max(A.offsets[e], 0), int(A.tokens)));
        hi = uint32_t(min(max(A.offsets[e + 1], int(lo)), int(A.tokens)));
    }
    if (hi == lo) return;  // the same for all blocks of a cluster
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < Shape::stages; ++s) {
            mbar_init(&c.full[s], 1 + 32);  // the records, and every lane's copies of x
            mbar_init(&c.empty[s], kGvWarps);
        }
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const uint8_t* stream = A.stream + e * A.stride;
    const uint32_t h = min(8u, L.blocks16 - b0);
    const uint32_t s0 = uint32_t(uint64_t(L.slices) * part / P.split);
    const uint32_t s1 = uint32_t(uint64_t(L.slices) * (part + 1) / P.split);
    const uint32_t tiles = (hi - lo + 8 * NT - 1) / (8 * NT);
    const Q4Masks mk = Q4Masks::make<HALF>();
    uint32_t n = 0;  // slices so far
    bool ok = true;
    for (uint32_t tile = 0; tile < tiles; ++tile) {
        const uint32_t t0 = lo + tile * 8 * NT;
        if (warp == kGvWarps) {  // producer; without a cluster it runs ahead into the next tiles
            const uint32_t ntok = min(8u * NT, hi - t0);
            for (uint32_t s = s0; ok && s < s1; ++s) {
                const uint32_t st = n % Shape::stages, round = n / Shape::stages;
                ok = round == 0 || gv_wait(&c.empty[st], (round - 1u) & 1u, c, A.status);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&c.full[st], h * L.rec);
                    bulk_load(w_ring + st * P.pitch, stream + q4_record(L, b0, s), h * L.rec,
                              &c.full[st]);
                }
                __syncwarp();
                const uint32_t dst = smem_addr(x_ring + st * Shape::x_bytes);
                if (P.x_bytes == 2) {
                    gv_copy_x<2>(P, dst, t0, ntok, s, lane);
                    mbar_arrive(&c.full[st]);
                } else {
                    if (P.x_bytes == 16)
                        gv_copy_x<16>(P, dst, t0, ntok, s, lane);
                    else if (P.x_bytes == 8)
                        gv_copy_x<8>(P, dst, t0, ntok, s, lane);
                    else
                        gv_copy_x<4>(P, dst, t0, ntok, s, lane);
                    // this lane's arrival, once its copies have landed
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                     smem_addr(&c.full[st]))
                                 : "memory");
                }
                ++n;
            }
        } else {
            float acc[NT][4] = {};
            for (uint32_t s = s0; ok && s < s1; ++s, ++n) {
                const uint32_t st = n % Shape::stages;
                ok = gv_wait(&c.full[st], (n / Shape::stages) & 1u, c, A.status);
                if (!ok) break;
                if (warp < h)
                    record_mma<HALF, NT, PER>(smem_addr(w_ring + st * P.pitch) + warp * L.rec,
                                              smem_addr(x_ring + st * Shape::x_bytes), L.zeros,
                                              L.half_scales, g, t, mk, acc);
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.empty[st]);
            }
            if (P.split == 1) {
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t row = (b0 + warp) * kQ4Rows + g + 8 * (j >> 1);
                        const uint32_t p = t0 + 8 * k + 2 * t + (j & 1);
                        if (ok && row < L.rows && p < hi) q4_store<HALF>(A, p, row, acc[k][j]);
                    }
            } else {  // (a warp that gave up has no sums: the results are NaN)
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sums[warp * Shape::vals + (k * 4 + j) * 32 + lane] =
                            ok ? acc[k][j] : __int_as_float(0x7FC00000);
            }
        }
        if (P.split > 1) {
            // each block adds and writes its share of the rows, over the blocks in order
            const cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            for (uint32_t v = part * kGvThreads + threadIdx.x; v < kGvWarps * Shape::vals;
                 v += P.split * kGvThreads) {
                const uint32_t r = v / Shape::vals, k = v % Shape::vals / 128, j = v % 128 / 32;
                const uint32_t gg = v % 32 / 4, tt = v % 4;
                const uint32_t row = (b0 + r) * kQ4Rows + gg + 8 * (j >> 1);
                const uint32_t p = t0 + 8 * k + 2 * tt + (j & 1);
                if (row >= L.rows || p >= hi) continue;
                float sum = 0.f;
                for (uint32_t q = 0; q < P.split; ++q) sum += cluster.map_shared_rank(sums, q)[v];
                q4_store<HALF>(A, p, row, sum);
            }
            cluster.sync();
        }
    }
    // No copy outlives the block, whichever warp gave up (bounded polls). Where none
    // did, the warps have waited for every copy.
    __syncthreads();
    if (warp == kGvWarps && c.abort) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        ring_last_fills(n, Shape::stages, [&](uint32_t st, uint32_t parity) {
            for (int j = 0; j < (1 << 16); ++j)
                if (__all_sync(0xFFFFFFFFu, gv_poll(&c.full[st], parity))) break;
        });
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) q4_check_header(stream, L, A.status);
}

template <bool HALF, int NT, int PER>
cudaError_t gv_launch(const GvParams& P, cudaStream_t stream) {
    static std::mutex mu;
    static bool set[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = q4_gemv_kernel<HALF, NT, PER>;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(gv_smem<NT>(8 * (kQ4Codes + 32 * 4 + 64))));
            if (err != cudaSuccess) return err;
            set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((P.L.blocks16 + 7) / 8 * P.split, P.a.experts);
    cfg.blockDim = dim3(kGvThreads);
    cfg.dynamicSmemBytes = gv_smem<NT>(P.pitch);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <bool HALF, int NT>
cudaError_t gv_per(const GvParams& P, cudaStream_t stream) {
    return P.L.per == 1   ? gv_launch<HALF, NT, 1>(P, stream)
           : P.L.per == 2 ? gv_launch<HALF, NT, 2>(P, stream)
                          : gv_launch<HALF, NT, 4>(P, stream);
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
    P.pitch = 8 * L.rec;
    const uint64_t al = reinterpret_cast<uintptr_t>(a.x) | (a.ldx * 2);
    P.x_bytes = al % 16 == 0 ? 16u : al % 8 == 0 ? 8u : al % 4 == 0 ? 4u : 2u;
    // Matrices that can have rows, and rows of x such a matrix has on average.
    const uint32_t used = a.offsets == nullptr ? 1u : a.tokens < a.experts ? a.tokens : a.experts;
    const uint32_t rows = (a.tokens + used - 1) / used;
    // As many blocks as are resident at a time (two a multiprocessor), if each
    // then has two slices or more.
    const uint64_t blocks = uint64_t(used) * ((L.blocks16 + 7) / 8);
    P.split = 1;
    while (P.split < 8 && blocks * P.split * 2 <= 2ull * uint32_t(sms) &&
           L.slices / (2 * P.split) >= 2)
        P.split *= 2;
    if (a.flags & kQ4XHalf) return rows > 8 ? gv_per<true, 2>(P, stream) : gv_per<true, 1>(P, stream);
    return rows > 8 ? gv_per<false, 2>(P, stream) : gv_per<false, 1>(P, stream);
}

}  // namespace wc
