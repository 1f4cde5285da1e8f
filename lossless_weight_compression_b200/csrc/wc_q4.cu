// wc_q4.cu -- 4-bit streams with group scales: quantizing a 16-bit matrix,
// packing given codes, and expanding a stream (sm_100a).
//
// One thread block of 8 warps per 128 rows x 128 columns, one warp per record
// of 16 rows: lane l holds columns 8 (l & 15) .. + 7 of row l >> 4 of a row
// pair, so a group of 32, 64 or 128 columns is 4, 8 or 16 neighbouring lanes
// and its range is reduced by shuffles; the eight records are put together in
// shared memory and leave as one contiguous run of 16-byte stores. Each weight
// is read once and each stream byte written once. Measured (14336 x 4096 BF16,
// groups of 128): quantizing 42 us, 3.5 TB/s of the 6.5 a copy moves, bound by
// instruction issue (0.79 a cycle, about 13 instructions a weight); expanding 27 us,
// 5.5 TB/s, from L2 or HBM, issue 0.79 as well. Both together 65 us (119 us with a
// division, a rintf and a conversion to int for each weight); 1000 x 4100 FP16,
// groups of 32 with zero points, 10 us (35 us while groups of zeros and a ragged
// last slice took the slow paths).
#include "wc_q4_core.cuh"

namespace wc {
namespace {

constexpr int kQ4Threads = 256;
constexpr uint32_t kMaxRec = kQ4Codes + 32u * 4u + 64u;  // group 32 with zero points

template <bool HALF>
__device__ __forceinline__ float to_float(uint16_t b) {
    return HALF ? __half2float(__ushort_as_half(b)) : __uint_as_float(uint32_t(b) << 16);
}

template <bool HALF>
__device__ __forceinline__ uint16_t from_float(float v) {
    return HALF ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Two values rounded to 16 bits, the first in the low half.
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t d;
    if (HALF)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}

// Eight consecutive 16-bit values of a row from column c, zeros past the end, as
// vectors V that divide the row's address and its length, so that each is inside
// or outside.
template <typename V>
__device__ __forceinline__ uint4 load8(const uint16_t* row, uint32_t c, uint32_t cols, bool live) {
    constexpr int N = 16 / sizeof(V);
    V v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = V{};
        if (live && c + 8 / N * k < cols) v[k] = __ldcs(reinterpret_cast<const V*>(row + c) + k);
    }
    uint4 u;
    memcpy(&u, v, 16);
    return u;
}

// Eight 16-bit values to a row from column c, up to the last column.
template <typename V>
__device__ __forceinline__ void store8(uint16_t* row, uint32_t c, uint32_t cols, uint4 u) {
    constexpr int N = 16 / sizeof(V);
    V v[N];
    memcpy(v, &u, 16);
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (c + 8 / N * k < cols) __stcs(reinterpret_cast<V*>(row + c) + k, v[k]);
}

// Adding and subtracting 1.5 * 2^23 rounds |x| < 2^22 to the nearest integer,
// ties to even, on the FMA pipe (rintf and conversions to int run at an eighth of
// its rate; with them and a division a weight that unit bound the kernel).
constexpr float kRound = 12582912.f;

__device__ __forceinline__ float approx_rcp(float s) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// w / s to within a rounding, and exactly where the quotient is a half-integer
// up to 32: t = w r with r near 1 / s is off by a few 2^-23 of itself; the
// remainder w - t s is exact by FMA (its bits lie between 2^-20 and 2^-35 of w,
// s having at most 11), and adding r times it (a Newton step on the remainder)
// leaves 2^-40 of the quotient before the last rounding, which a quotient that
// FP32 holds absorbs. So the quotient rounds to the integer that the exact one
// rounds to: with s = S 2^b and w = W 2^a, W and S of equal length below 2^11, it
// is a half-integer or at least 2^-13 away from each: w / s - (2 k + 1) / 2 =
// (2 W 2^(a-b) - (2 k + 1) S) / (2 S), whose numerator is a multiple of 1/2 where
// w / s is near 1/2 or above (a - b >= -2).
__device__ __forceinline__ float quotient(float w, float s, float r) {
    const float t = w * r;
    return fmaf(fmaf(-t, s, w), r, t);
}

// The larger (smaller) of two pairs of 16-bit floats; NaN if either is.
template <bool HALF>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (HALF)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <bool HALF>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (HALF)
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The word of eight codes in element order.
__device__ __forceinline__ uint32_t pack8(const uint32_t (&q)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= q[e] << (4 * ((e >> 1) + 4 * (e & 1)));
    return w;
}

// The block's records from shared memory to the stream.
__device__ __forceinline__ void store_records(uint8_t* dst, const uint8_t* sm, uint32_t bytes) {
    __syncthreads();
    for (uint32_t k = threadIdx.x * 16u; k < bytes; k += kQ4Threads * 16u)
        *reinterpret_cast<uint4*>(dst + k) = *reinterpret_cast<const uint4*>(sm + k);
}

__device__ __forceinline__ void store_header(const Q4Layout& L, uint8_t* out) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 16)
        reinterpret_cast<uint64_t*>(out)[threadIdx.x] = q4_header_word(L, threadIdx.x);
}

// Scale, zero point and codes of each group, round to nearest even throughout:
//   without zero points  s = rnd16(max|w| / 7), q = clamp(rint(w / s), -8, 7) + 8
//   with zero points     lo = min(w, 0), hi = max(w, 0), s = rnd16((hi - lo) / 15),
//                        z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(w / s) + z, 0, 15)
// (s = 0: every code stands for zero). The range is reduced as one pair of 16-bit
// floats a lane, max(w, 0) and max(-w, 0); the codes of four elements add up as
// 16^k-weighted floats (below 2^16, exact).
//
// A scale whose reciprocal FP32 cannot hold, infinities or NaN: the definition's
// steps as they stand. Not inlined: the eight row pairs of a warp
// are straight-line code, and every warp passes through all of it.
template <bool HALF>
__device__ __noinline__ uint32_t odd_group(uint4 v, float sc, float lo, float& z, bool zeros) {
    const float d = sc > 0.f ? sc : 1.f;
    if (zeros) z = fminf(fmaxf(rintf(lo / d), 0.f), 15.f);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = to_float<HALF>(uint16_t(u[e >> 1] >> (16 * (e & 1))));
        q[e] = uint32_t(fminf(fmaxf(rintf(f / d) + z, 0.f), 15.f));
    }
    return pack8(q);
}

template <bool HALF, bool ZEROS, int PER>
__global__ void __launch_bounds__(kQ4Threads)
    q4_quantize_kernel(const uint16_t* __restrict__ w, uint64_t ld, Q4Layout L, uint32_t vec,
                       uint8_t* __restrict__ out) {
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int kLanes = 16 / PER;  // of a group
    constexpr float kSteps = ZEROS ? 15.f : 7.f, kInv = 1.f / kSteps;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t b0 = blockIdx.y * 8, s = blockIdx.x;
    const uint32_t h = min(8u, L.blocks16 - b0);
    store_header(L, out);
    if (warp < h) {
        uint8_t* rec = sm + warp * L.rec;
        const uint32_t c8 = lane & 15u, c = s * kQ4Cols + 8 * c8;
        const uint32_t row0 = (b0 + warp) * kQ4Rows + (lane >> 4);
        const uint16_t* p = w + uint64_t(row0) * ld;
        uint4 v[8];
        auto load = [&](auto vector) {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
                v[k] = load8<decltype(vector)>(p + uint64_t(2 * k) * ld, c, L.cols,
                                               row0 + 2 * k < L.rows);
        };
        if (vec == 16)
            load(uint4());
        else if (vec == 8)
            load(uint2());
        else if (vec == 4)
            load(uint32_t());
        else
            load(static_cast<unsigned short>(0));
        const uint32_t at = (c8 & 3u) * 256 + (lane >> 4) * 16 + (c8 >> 2) * 4;
        const bool first = (c8 & (kLanes - 1)) == 0;  // of its group
        uint8_t* meta = rec + kQ4Codes + (c8 / kLanes * 16 + (lane >> 4)) * 2;
        uint8_t* zmeta = rec + kQ4Codes + 32 * PER + c8 / kLanes * 16 + (lane >> 4);
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            const uint32_t mx = max2<HALF>(max2<HALF>(u[0], u[1]), max2<HALF>(u[2], u[3]));
            const uint32_t mn = min2<HALF>(min2<HALF>(u[0], u[1]), min2<HALF>(u[2], u[3])) ^
                                0x80008000u;  // negated: the largest -w
            // {even w, even -w} against {odd w, odd -w}, and 0
            uint32_t m = max2<HALF>(prmt(mx, mn, 0x5410u), prmt(mx, mn, 0x7632u));
            m = max2<HALF>(m, 0u);
#pragma unroll
            for (int o = 1; o < kLanes; o *= 2)
                m = max2<HALF>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float hi = to_float<HALF>(uint16_t(m)), lo = to_float<HALF>(uint16_t(m >> 16));
            // (a NaN made both NaN; infinities of both signs count as one)
            const float inf = __int_as_float(0x7F800000);
            float range = ZEROS ? hi + lo : fmaxf(hi, lo);
            if (hi != hi || (hi == inf && lo == inf)) range = __int_as_float(0x7FC00000);
            // range / steps, again by a Newton step on the remainder: the nearest FP32
            // value of the quotient, which lies 1/14 (1/30) of a step or more from the
            // middle of two. Infinities and NaN, whose remainder is NaN, stay as they are.
            const float t0 = range * kInv;
            const float t1 = fmaf(fmaf(-t0, kSteps, range), kInv, t0);
            const uint16_t sbits = from_float<HALF>(range < inf ? t1 : range);
            const float sc = to_float<HALF>(sbits);
            uint32_t word;
            float z = 8.f;
            if (sc == 0.f) {  // every code stands for zero
                z = ZEROS ? 0.f : 8.f;
                word = ZEROS ? 0u : 0x88888888u;
            } else if (__builtin_expect(sc > 1e-30f && sc < 1e30f, 1)) {
                const float r = approx_rcp(sc);
                if (ZEROS) z = fminf((quotient(lo, sc, r) + kRound) - kRound, 15.f);
                const float zk = z - kRound, top = 15.f - z;
                float part[2] = {0.f, 0.f};  // even and odd elements
#pragma unroll
                for (int e = 7; e >= 0; --e) {
                    const float f = HALF ? to_float<HALF>(uint16_t(u[e >> 1] >> (16 * (e & 1))))
                                         : __uint_as_float(e & 1 ? u[e >> 1] & 0xFFFF0000u : u[e >> 1] << 16);
                    // clamped before the rounding: the bounds are integers
                    const float t = fminf(fmaxf(quotient(f, sc, r), -z), top);
                    part[e & 1] = fmaf(part[e & 1], 16.f, (t + kRound) + zk);
                }
                word = prmt(__float_as_uint(part[0] + 8388608.f), __float_as_uint(part[1] + 8388608.f),
                            0x5410u);
            } else {
                word = odd_group<HALF>(v[k], sc, lo, z, ZEROS);
            }
            *reinterpret_cast<uint32_t*>(rec + at + k * 32) = word;
            if (first) {
                *reinterpret_cast<uint16_t*>(meta + k * 4) = sbits;
                if (ZEROS) zmeta[k * 2] = uint8_t(z);
            }
        }
        if (ZEROS && PER == 1 && lane < 16) rec[kQ4Codes + 32 + 16 + lane] = 0;  // padding
    }
    store_records(out + q4_record(L, b0, s), sm, h * L.rec);
}

template <bool HALF, bool ZEROS>
auto quantize_by_group(uint32_t per) {
    return per == 1   ? q4_quantize_kernel<HALF, ZEROS, 1>
           : per == 2 ? q4_quantize_kernel<HALF, ZEROS, 2>
                      : q4_quantize_kernel<HALF, ZEROS, 4>;
}

__global__ void __launch_bounds__(kQ4Threads)
    q4_pack_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                   const uint8_t* __restrict__ zeros, Q4Layout L, uint8_t* __restrict__ out) {
    extern __shared__ __align__(16) uint8_t sm[];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t b0 = blockIdx.y * 8, s = blockIdx.x;
    const uint32_t h = min(8u, L.blocks16 - b0);
    const uint32_t groups = uint32_t((uint64_t(L.cols) + L.group - 1) / L.group);
    store_header(L, out);
    if (warp < h) {
        uint8_t* rec = sm + warp * L.rec;
        const uint32_t c8 = lane & 15u, c = s * kQ4Cols + 8 * c8;
        const uint32_t g = c8 / (L.group / 8), gg = s * L.per + g;
        for (uint32_t k = 0; k < 8; ++k) {
            const uint32_t r = 2 * k + (lane >> 4), row = (b0 + warp) * kQ4Rows + r;
            const bool live = row < L.rows;
            const bool has = live && gg < groups;
            const uint32_t z = !L.zeros ? 8u : has ? zeros[uint64_t(row) * groups + gg] & 15u : 0u;
            uint32_t q[8];
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                q[e] = live && c + e < L.cols ? codes[uint64_t(row) * L.cols + c + e] & 15u : z;
            *reinterpret_cast<uint32_t*>(rec + (c8 & 3u) * 256 + r * 16 + (c8 >> 2) * 4) = pack8(q);
            if ((c8 & (L.group / 8 - 1)) == 0) {
                *reinterpret_cast<uint16_t*>(rec + kQ4Codes + (g * 16 + r) * 2) =
                    has ? scales[uint64_t(row) * groups + gg] : uint16_t(0);
                if (L.zeros) rec[kQ4Codes + 32 * L.per + g * 16 + r] = uint8_t(z);
            }
        }
        if (L.zeros && L.per == 1 && lane < 16) rec[kQ4Codes + 32 + 16 + lane] = 0;  // padding
    }
    store_records(out + q4_record(L, b0, s), sm, h * L.rec);
}

// s (q - z) in FP32 is exact (at most 11 + 4 bits); one rounding to 16 bits.
template <int DT>
__global__ void __launch_bounds__(kQ4Threads)
    q4_dequantize_kernel(const uint8_t* __restrict__ in, Q4Layout L, void* __restrict__ out,
                         uint64_t ld, uint32_t vec, int32_t* status) {
    extern __shared__ __align__(16) uint8_t sm[];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t b0 = blockIdx.y * 8, s = blockIdx.x;
    const uint32_t h = min(8u, L.blocks16 - b0);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) q4_check_header(in, L, status);
    const uint8_t* src = in + q4_record(L, b0, s);
    for (uint32_t k = threadIdx.x * 16u; k < h * L.rec; k += kQ4Threads * 16u)
        *reinterpret_cast<uint4*>(sm + k) = ld_stream_v4(src + k);
    __syncthreads();
    if (warp >= h) return;
    const uint8_t* rec = sm + warp * L.rec;
    const uint32_t c8 = lane & 15u, c = s * kQ4Cols + 8 * c8;
    const uint32_t g = c8 / (L.group / 8);
    if (c >= L.cols) return;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
        const uint32_t r = 2 * k + (lane >> 4), row = (b0 + warp) * kQ4Rows + r;
        if (row >= L.rows) continue;
        const uint32_t word =
            *reinterpret_cast<const uint32_t*>(rec + (c8 & 3u) * 256 + r * 16 + (c8 >> 2) * 4);
        const float sc = q4_scale(*reinterpret_cast<const uint16_t*>(rec + kQ4Codes + (g * 16 + r) * 2),
                                  L.half_scales);
        // 2^23 + q and 2^23 + z in the low mantissa bits: their difference is q - z
        const float z = __uint_as_float(
            0x4B000000u | (L.zeros ? rec[kQ4Codes + 32 * L.per + g * 16 + r] & 15u : 8u));
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = sc * (__uint_as_float(((word >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u) | 0x4B000000u) - z);
        if (DT == 2) {
            float* o = static_cast<float*>(out) + uint64_t(row) * ld + c;
            if (vec == 16 && c + 8 <= L.cols) {
                st_stream_v4(o, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                           __float_as_uint(f[2]), __float_as_uint(f[3])));
                st_stream_v4(o + 4, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                               __float_as_uint(f[6]), __float_as_uint(f[7])));
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e)
                    if (c + e < L.cols) o[e] = f[e];
            }
        } else {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = pack2<DT == 1>(f[2 * e], f[2 * e + 1]);
            uint16_t* o = static_cast<uint16_t*>(out) + uint64_t(row) * ld;
            const uint4 u = make_uint4(b[0], b[1], b[2], b[3]);
            if (vec == 16)
                store8<uint4>(o, c, L.cols, u);
            else if (vec == 8)
                store8<uint2>(o, c, L.cols, u);
            else if (vec == 4)
                store8<uint32_t>(o, c, L.cols, u);
            else
                store8<unsigned short>(o, c, L.cols, u);
        }
    }
}

// Bytes (2 to 16) that divide the address and the length of every row.
uint32_t row_align(const void* p, uint64_t ld, uint64_t cols, uint32_t size) {
    const uint64_t a = reinterpret_cast<uintptr_t>(p) | (ld * size) | (cols * size);
    return a % 16 == 0 ? 16u : a % 8 == 0 ? 8u : a % 4 == 0 ? 4u : 2u;
}

dim3 q4_grid(const Q4Layout& L) { return dim3(L.slices, (L.blocks16 + 7) / 8); }

// An empty matrix is a bare header.
__global__ void q4_header_kernel(Q4Layout L, uint8_t* out) { store_header(L, out); }

}  // namespace

cudaError_t launch_q4_quantize(const void* w, uint64_t ld, const Q4Layout& L, uint8_t* out,
                               cudaStream_t stream) {
    if (L.blocks16 == 0) {
        q4_header_kernel<<<1, 32, 0, stream>>>(L, out);
        return cudaGetLastError();
    }
    const auto kernel =
        L.half_scales
            ? (L.zeros ? quantize_by_group<true, true>(L.per) : quantize_by_group<true, false>(L.per))
            : (L.zeros ? quantize_by_group<false, true>(L.per) : quantize_by_group<false, false>(L.per));
    kernel<<<q4_grid(L), kQ4Threads, 8 * kMaxRec, stream>>>(static_cast<const uint16_t*>(w), ld, L,
                                                            row_align(w, ld, L.cols, 2), out);
    return cudaGetLastError();
}

cudaError_t launch_q4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros,
                           const Q4Layout& L, uint8_t* out, cudaStream_t stream) {
    if (L.blocks16 == 0) {
        q4_header_kernel<<<1, 32, 0, stream>>>(L, out);
        return cudaGetLastError();
    }
    q4_pack_kernel<<<q4_grid(L), kQ4Threads, 8 * kMaxRec, stream>>>(
        codes, static_cast<const uint16_t*>(scales), zeros, L, out);
    return cudaGetLastError();
}

cudaError_t launch_q4_dequantize(const uint8_t* in, const Q4Layout& L, void* out, uint64_t ld,
                                 uint32_t dtype, int32_t* status, cudaStream_t stream) {
    if (L.blocks16 == 0) return cudaSuccess;
    const auto kernel = dtype == 2   ? q4_dequantize_kernel<2>
                        : dtype == 1 ? q4_dequantize_kernel<1>
                                     : q4_dequantize_kernel<0>;
    kernel<<<q4_grid(L), kQ4Threads, 8 * kMaxRec, stream>>>(in, L, out, ld,
                                                            row_align(out, ld, L.cols, dtype == 2 ? 4 : 2), status);
    return cudaGetLastError();
}

}  // namespace wc
