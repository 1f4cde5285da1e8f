// wc_moe.cu -- rows of activations sorted by expert and back, and the
// gradients (sm_100a). A slot is one (token, choice) pair; `inverse` holds each
// slot's row in the sorted matrix, a value outside 0..rows-1 meaning none.
//
// All but the sort move each row once: a token's row is read once and written to
// its slots' rows, or its slots' rows are read and summed, with 16-byte accesses
// where the rows allow them. Measured (BF16; beside it the bytes at the copy's
// rate): 16,384 tokens x 6 slots of 4 KB rows: gather 77 us (73), its gradient 79
// us (73), sort 19 us; 8192 tokens x 2 slots of 8 KB rows: combine 40 us (31), its
// backward 57 us (52).
#include <cooperative_groups.h>

#include <mutex>

#include "wc_q4_core.cuh"

namespace wc {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Counting sort of the slots by expert, stable: row = first row of the expert +
// earlier slots of the same expert. One cluster of up to 8 blocks: each warp
// owns consecutive slots and counts them in its own histogram (the lanes of one
// expert found by a ballot per bit of the id, so no atomics); the histograms are
// scanned over the block's
// warps, the cluster's blocks (through distributed shared memory) and the
// experts; then each warp adds the sums to its slots' ranks. No workspace and one
// launch. The counting is bound by instruction issue on the cluster's eight
// multiprocessors (98,304 slots: 19 us), far below the row copies that follow.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr uint32_t kMaxExperts = 1024;

// Lanes of the warp whose id equals this lane's (ids < 2^bits).
__device__ __forceinline__ uint32_t same_id(uint32_t id, int bits) {
    uint32_t m = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, (id >> b) & 1u);
        m &= (id >> b) & 1u ? set : ~set;
    }
    return m;
}

constexpr int kSortBatch = 8;  // ids of a lane loaded ahead of the dependent counting

__global__ void __launch_bounds__(kSortThreads)
    moe_sort_kernel(const int32_t* __restrict__ ids, uint32_t slots, uint32_t experts,
                    int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                    int32_t* inverse) {
    extern __shared__ uint32_t sm[];
    uint32_t* hist = sm;                            // [warps][experts]
    uint32_t* total = sm + kSortWarps * experts;    // [experts] of this block
    uint32_t* base = total + experts;               // [experts] first row for this block
    __shared__ uint32_t warp_sum[kSortWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t nblk = gridDim.x, blk = blockIdx.x;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint64_t workers = uint64_t(nblk) * kSortWarps;
    const uint32_t per = uint32_t((slots + workers * 32 - 1) / (workers * 32)) * 32;
    const uint64_t first = uint64_t(blk * kSortWarps + warp) * per;
    const uint32_t begin = uint32_t(first < slots ? first : slots);
    const uint32_t end = uint32_t(first + per < slots ? first + per : slots);
    uint32_t* mine = hist + warp * experts;
    for (uint32_t k = tid; k < kSortWarps * experts; k += kSortThreads) hist[k] = 0;
    __syncthreads();
    const int bits = 32 - __clz(int(experts));  // ids and the dropped ones' `experts`
    const uint32_t below = (1u << lane) - 1u;
    for (uint32_t s0 = begin; s0 < end; s0 += 32 * kSortBatch) {
        uint32_t id[kSortBatch];
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k)
            id[k] = s0 + 32 * k + lane < end ? min(uint32_t(ids[s0 + 32 * k + lane]), experts)
                                             : experts;
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k) {
            const uint32_t s = s0 + 32 * k + lane;
            if (s0 + 32 * k >= end) break;
            const uint32_t same = same_id(id[k], bits);
            // the slot's rank among the warp's of its expert waits in `inverse`
            if (s < end)
                inverse[s] = id[k] < experts ? int32_t(mine[id[k]] + __popc(same & below)) : -1;
            __syncwarp();
            if (id[k] < experts && (same & below) == 0) mine[id[k]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (uint32_t e = tid; e < experts; e += kSortThreads) {
        uint32_t run = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t v = hist[w * experts + e];
            hist[w * experts + e] = run;
            run += v;
        }
        total[e] = run;
    }
    cluster.sync();
    // thread e: the expert's slots in earlier blocks and in all blocks
    uint32_t before = 0, all = 0;
    if (tid < experts)
        for (uint32_t b = 0; b < nblk; ++b) {
            const uint32_t v = cluster.map_shared_rank(total, b)[tid];
            before += b < blk ? v : 0u;
            all += v;
        }
    uint32_t incl = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= uint32_t(o)) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    cluster.sync();  // also: every block has read the totals
    uint32_t ahead = 0;
    for (uint32_t w = 0; w < warp; ++w) ahead += warp_sum[w];
    const uint32_t begins = ahead + incl - all;
    if (tid < experts) {
        base[tid] = begins + before;
        if (blk == 0) {
            offsets[tid] = int32_t(begins);
            if (tid == experts - 1) offsets[experts] = int32_t(begins + all);
        }
    }
    uint32_t rows = 0;
    for (int w = 0; w < kSortWarps; ++w) rows += warp_sum[w];
    __syncthreads();
    for (uint32_t s0 = begin + lane; s0 < end; s0 += 32 * kSortBatch) {
        int32_t id[kSortBatch], pos[kSortBatch];
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k)
            if (s0 + 32 * k < end) {
                id[k] = ids[s0 + 32 * k];
                pos[k] = inverse[s0 + 32 * k];  // written by this thread
            }
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k) {
            const uint32_t s = s0 + 32 * k;
            if (s >= end) break;
            if (pos[k] >= 0) {
                pos[k] += int32_t(base[id[k]] + mine[id[k]]);
                inverse[s] = pos[k];
                if (order != nullptr) order[pos[k]] = int32_t(s);
            }
            if (order != nullptr && s >= rows) order[s] = -1;
        }
    }
}

// ---------------------------------------------------------------------------
// Row copies and sums. VEC: the widest vector that every row's address allows.
// A warp owns a segment of a token's row: kUnroll vectors a lane.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int kUnroll = 4;

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ float to(__half v) { return __half2float(v); }
    static __device__ __half from(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
    static __device__ float to(float v) { return v; }
    static __device__ float from(float v) { return v; }
};

template <typename T, typename V>
__device__ __forceinline__ void unpack(const V& v, float (&f)[sizeof(V) / sizeof(T)]) {
    T t[sizeof(V) / sizeof(T)];
    memcpy(t, &v, sizeof(V));
#pragma unroll
    for (int k = 0; k < int(sizeof(V) / sizeof(T)); ++k) f[k] = Elem<T>::to(t[k]);
}

template <typename T, typename V>
__device__ __forceinline__ V pack(const float (&f)[sizeof(V) / sizeof(T)]) {
    T t[sizeof(V) / sizeof(T)];
#pragma unroll
    for (int k = 0; k < int(sizeof(V) / sizeof(T)); ++k) t[k] = Elem<T>::from(f[k]);
    V v;
    memcpy(&v, t, sizeof(V));
    return v;
}

// A read of data used once: not kept in L1.
template <typename V>
__device__ __forceinline__ V ldg_stream(const V* p) {
    return __ldcs(p);
}
template <>
__device__ __forceinline__ uint16_t ldg_stream<uint16_t>(const uint16_t* p) {
    return __ldcs(reinterpret_cast<const unsigned short*>(p));
}

struct RowParams {
    uint64_t tokens, rows;
    uint32_t top;
    uint32_t nvec;      // vectors of a row
    uint32_t segs;      // segments of a row
    uint32_t team;      // backward: threads of a token
    const int32_t* inverse;
};

template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    moe_gather_kernel(RowParams P, const uint8_t* __restrict__ x, uint64_t ldx,
                      uint8_t* __restrict__ out, uint64_t ldo) {
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t unit = (uint64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
    const uint64_t tok = unit / P.segs;
    if (tok >= P.tokens) return;
    const uint32_t v0 = uint32_t(unit % P.segs) * (32 * kUnroll) + lane;
    const V* src = reinterpret_cast<const V*>(x + tok * ldx);
    V v[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
        if (v0 + 32 * k < P.nvec) v[k] = src[v0 + 32 * k];
    for (uint32_t j = 0; j < P.top; ++j) {
        const int32_t p = P.inverse[tok * P.top + j];
        if (p < 0 || uint64_t(p) >= P.rows) continue;
        V* dst = reinterpret_cast<V*>(out + uint64_t(p) * ldo);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (v0 + 32 * k < P.nvec) dst[v0 + 32 * k] = v[k];
    }
}

// Slots are taken AHEAD at a time, UNROLL vectors a lane of each, all on their way
// before the first is used (a slot without a row loads nothing and adds nothing):
// one slot after the other left the memory waiting for indices (16,384 tokens of
// 6 rows of 4 KB: 186 us, so 75, where the bytes take 67).
template <typename T, typename V, int AHEAD, int UNROLL>
__global__ void __launch_bounds__(kRowThreads)
    moe_combine_kernel(RowParams P, const uint8_t* __restrict__ y, uint64_t ldy,
                       const float* __restrict__ weights, uint8_t* __restrict__ out, uint64_t ldo) {
    constexpr int N = sizeof(V) / sizeof(T);
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t unit = (uint64_t(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
    const uint64_t tok = unit / P.segs;
    if (tok >= P.tokens) return;
    const uint32_t v0 = uint32_t(unit % P.segs) * (32 * UNROLL) + lane;
    float acc[UNROLL][N] = {};
    for (uint32_t j0 = 0; j0 < P.top; j0 += AHEAD) {
        int32_t p[AHEAD];
        float w[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            p[j] = j0 + j < P.top ? P.inverse[tok * P.top + j0 + j] : -1;
            if (p[j] >= 0 && uint64_t(p[j]) >= P.rows) p[j] = -1;
            w[j] = weights != nullptr && p[j] >= 0 ? weights[tok * P.top + j0 + j] : 1.f;
        }
        V v[AHEAD][UNROLL];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
#pragma unroll
            for (int k = 0; k < UNROLL; ++k)
                if (p[j] >= 0 && v0 + 32 * k < P.nvec)
                    v[j][k] = ldg_stream(reinterpret_cast<const V*>(y + uint64_t(p[j]) * ldy) + v0 + 32 * k);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (p[j] < 0) continue;
#pragma unroll
            for (int k = 0; k < UNROLL; ++k)
                if (v0 + 32 * k < P.nvec) {
                    float f[N];
                    unpack<T, V>(v[j][k], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[k][i] = fmaf(w[j], f[i], acc[k][i]);
                }
        }
    }
    V* dst = reinterpret_cast<V*>(out + tok * ldo);
#pragma unroll
    for (int k = 0; k < UNROLL; ++k)
        if (v0 + 32 * k < P.nvec) dst[v0 + 32 * k] = pack<T, V>(acc[k]);
}

// dy[p] = w * dout[token] and dw = <dout[token], y[p]> of each slot: P.team
// threads (32 to 256) own a token, so that dout is read once and each product's
// sum stays in registers until one reduction in a fixed order. Slots are taken
// SLOTS at a time, with kBwUnroll vectors of each on their way.
constexpr int kBwUnroll = 2;

template <typename T, typename V, int SLOTS>
__global__ void __launch_bounds__(kRowThreads)
    moe_combine_backward_kernel(RowParams P, const uint8_t* __restrict__ dout, uint64_t ldd,
                                const uint8_t* __restrict__ y, uint64_t ldy,
                                const float* __restrict__ weights, uint8_t* __restrict__ dy,
                                uint64_t lddy, float* __restrict__ dweights) {
    constexpr int N = sizeof(V) / sizeof(T);
    __shared__ float red[SLOTS][kRowThreads / 32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t tid = threadIdx.x % P.team;
    const uint64_t tok = uint64_t(blockIdx.x) * (kRowThreads / P.team) + threadIdx.x / P.team;
    const bool live = tok < P.tokens;  // (every thread reaches the barriers)
    const V* d = reinterpret_cast<const V*>(dout + tok * ldd);
    for (uint32_t j0 = 0; j0 < P.top; j0 += SLOTS) {
        int32_t p[SLOTS];
        float w[SLOTS], dot[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            dot[j] = 0.f;
            w[j] = 1.f;
            p[j] = -1;
            if (live && j0 + j < P.top) {
                p[j] = P.inverse[tok * P.top + j0 + j];
                if (p[j] >= 0 && uint64_t(p[j]) >= P.rows) p[j] = -1;
                if (weights != nullptr) w[j] = weights[tok * P.top + j0 + j];
            }
        }
        if (live) {
            for (uint32_t v0 = tid; v0 < P.nvec; v0 += kBwUnroll * P.team) {
                V dv[kBwUnroll], yv[SLOTS][kBwUnroll];
#pragma unroll
                for (int k = 0; k < kBwUnroll; ++k) {
                    const uint32_t v = v0 + k * P.team;
                    if (v >= P.nvec) continue;
                    dv[k] = d[v];
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j)
                        if (p[j] >= 0)
                            yv[j][k] = ldg_stream(reinterpret_cast<const V*>(y + uint64_t(p[j]) * ldy) + v);
                }
#pragma unroll
                for (int k = 0; k < kBwUnroll; ++k) {
                    const uint32_t v = v0 + k * P.team;
                    if (v >= P.nvec) continue;
                    float df[N];
                    unpack<T, V>(dv[k], df);
#pragma unroll
                    for (int j = 0; j < SLOTS; ++j) {
                        if (p[j] < 0) continue;
                        float f[N];
                        unpack<T, V>(yv[j][k], f);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            dot[j] = fmaf(df[i], f[i], dot[j]);
                            f[i] = w[j] * df[i];
                        }
                        reinterpret_cast<V*>(dy + uint64_t(p[j]) * lddy)[v] = pack<T, V>(f);
                    }
                }
            }
        }
        if (dweights != nullptr) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o /= 2) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
                if (lane == 0) red[j][warp] = dot[j];
            }
            __syncthreads();
            if (live && tid < SLOTS && j0 + tid < P.top) {
                const uint32_t w0 = threadIdx.x / P.team * (P.team / 32);
                float sum = 0.f;
                for (uint32_t k = 0; k < P.team / 32; ++k) sum += red[tid][w0 + k];
                dweights[tok * P.top + j0 + tid] = sum;
            }
            __syncthreads();
        }
    }
}

uint32_t elem_size(uint32_t dtype) { return dtype == 2 ? 4u : 2u; }

// The widest vector (bytes) that divides every row's address and length.
uint32_t vec_bytes(uint64_t a, uint32_t size) {
    uint32_t v = 16;
    while (v > size && a % v != 0) v /= 2;
    return v;
}

cudaError_t too_large() { return cudaErrorInvalidValue; }

// Calls f(T{}, V{}) for the element type and the vector width.
template <typename F>
cudaError_t by_type(uint32_t dtype, uint32_t v, F f) {
    if (dtype == 2) {
        if (v == 16) return f(float(), uint4());
        if (v == 8) return f(float(), uint2());
        return f(float(), uint32_t());
    }
    if (dtype == 1) {
        if (v == 16) return f(__half(), uint4());
        if (v == 8) return f(__half(), uint2());
        if (v == 4) return f(__half(), uint32_t());
        return f(__half(), uint16_t());
    }
    if (v == 16) return f(__nv_bfloat16(), uint4());
    if (v == 8) return f(__nv_bfloat16(), uint2());
    if (v == 4) return f(__nv_bfloat16(), uint32_t());
    return f(__nv_bfloat16(), uint16_t());
}

RowParams row_params(const MoeArgs& a, uint32_t v, int unroll = kUnroll) {
    RowParams P;
    P.tokens = a.tokens;
    P.rows = a.rows;
    P.top = a.top;
    P.nvec = uint32_t(a.cols * elem_size(a.dtype) / v);
    P.segs = (P.nvec + 32 * unroll - 1) / (32 * unroll);
    P.team = 32;
    P.inverse = a.inverse;
    return P;
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t* ids, uint32_t slots, uint32_t experts, int32_t* offsets,
                            int32_t* order, int32_t* inverse, cudaStream_t stream) {
    static std::mutex mu;
    static bool set[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            err = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int((kSortWarps + 2) * kMaxExperts * 4));
            if (err != cudaSuccess) return err;
            set[dev] = true;
        }
    }
    const uint32_t want = (slots + 4095) / 4096;
    const uint32_t nblk = want < 1 ? 1 : want > 8 ? 8 : want;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nblk);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = (kSortWarps + 2) * experts * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nblk;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel, ids, slots, experts, offsets, order, inverse);
}

cudaError_t launch_moe_gather(const MoeArgs& a, const void* x, uint64_t ldx, void* out,
                              uint64_t ldo, cudaStream_t stream) {
    if (a.tokens == 0 || a.top == 0 || a.cols == 0 || a.rows == 0) return cudaSuccess;
    const uint32_t es = elem_size(a.dtype);
    const uint32_t v = vec_bytes(reinterpret_cast<uintptr_t>(x) | (ldx * es) |
                                     reinterpret_cast<uintptr_t>(out) | (ldo * es) | (a.cols * es),
                                 es);
    const RowParams P = row_params(a, v);
    const uint64_t blocks = (a.tokens * P.segs * 32 + kRowThreads - 1) / kRowThreads;
    if (blocks > 0x7FFFFFFFull) return too_large();
    const uint8_t* xs = static_cast<const uint8_t*>(x);
    uint8_t* os = static_cast<uint8_t*>(out);
    const dim3 grid = dim3(uint32_t(blocks));
    if (v == 16)
        moe_gather_kernel<uint4><<<grid, kRowThreads, 0, stream>>>(P, xs, ldx * es, os, ldo * es);
    else if (v == 8)
        moe_gather_kernel<uint2><<<grid, kRowThreads, 0, stream>>>(P, xs, ldx * es, os, ldo * es);
    else if (v == 4)
        moe_gather_kernel<uint32_t><<<grid, kRowThreads, 0, stream>>>(P, xs, ldx * es, os, ldo * es);
    else
        moe_gather_kernel<uint16_t><<<grid, kRowThreads, 0, stream>>>(P, xs, ldx * es, os, ldo * es);
    return cudaGetLastError();
}

cudaError_t launch_moe_combine(const MoeArgs& a, const void* y, uint64_t ldy, const float* weights,
                               void* out, uint64_t ldo, cudaStream_t stream) {
    if (a.tokens == 0 || a.cols == 0) return cudaSuccess;
    const uint32_t es = elem_size(a.dtype);
    const uint32_t v = vec_bytes(reinterpret_cast<uintptr_t>(y) | (ldy * es) |
                                     reinterpret_cast<uintptr_t>(out) | (ldo * es) | (a.cols * es),
                                 es);
    // Eight vectors a lane on their way where there are rows enough to fill the
    // machine so, as the slots have it; one of each slot where there are few.
    const uint64_t vectors = a.tokens * (a.cols * es / v);
    const int unroll = vectors < (1u << 19) ? 1 : a.top <= 2 ? 4 : 2;
    const RowParams P = row_params(a, v, unroll);
    const uint64_t blocks = (a.tokens * P.segs * 32 + kRowThreads - 1) / kRowThreads;
    if (blocks > 0x7FFFFFFFull) return too_large();
    return by_type(a.dtype, v, [&](auto t, auto vec) {
        using T = decltype(t);
        using V = decltype(vec);
        const auto kernel = unroll == 4   ? moe_combine_kernel<T, V, 2, 4>
                            : unroll == 2 ? moe_combine_kernel<T, V, 4, 2>
                                          : moe_combine_kernel<T, V, 4, 1>;
        kernel<<<uint32_t(blocks), kRowThreads, 0, stream>>>(P, static_cast<const uint8_t*>(y),
                                                             ldy * es, weights,
                                                             static_cast<uint8_t*>(out), ldo * es);
        return cudaGetLastError();
    });
}

cudaError_t launch_moe_combine_backward(const MoeArgs& a, const void* dout, uint64_t ldd,
                                        const void* y, uint64_t ldy, const float* weights,
                                        void* dy, uint64_t lddy, float* dweights,
                                        cudaStream_t stream) {
    if (a.tokens == 0 || a.top == 0) return cudaSuccess;
    const uint32_t es = elem_size(a.dtype);
    const uint32_t v = vec_bytes(reinterpret_cast<uintptr_t>(dout) | (ldd * es) |
                                     reinterpret_cast<uintptr_t>(y) | (ldy * es) |
                                     reinterpret_cast<uintptr_t>(dy) | (lddy * es) | (a.cols * es),
                                 es);
    RowParams P = row_params(a, v);
    while (P.team < uint32_t(kRowThreads) && P.team * kBwUnroll < P.nvec) P.team *= 2;
    const uint64_t per = kRowThreads / P.team;
    const uint64_t blocks = (a.tokens + per - 1) / per;
    if (blocks > 0x7FFFFFFFull) return too_large();
    return by_type(a.dtype, v, [&](auto t, auto vec) {
        using T = decltype(t);
        using V = decltype(vec);
        const auto kernel = a.top <= 2 ? moe_combine_backward_kernel<T, V, 2>
                                       : moe_combine_backward_kernel<T, V, 4>;
        kernel<<<uint32_t(blocks), kRowThreads, 0, stream>>>(
            P, static_cast<const uint8_t*>(dout), ldd * es, static_cast<const uint8_t*>(y), ldy * es,
            weights, static_cast<uint8_t*>(dy), lddy * es, dweights);
        return cudaGetLastError();
    });
}

}  // namespace wc
