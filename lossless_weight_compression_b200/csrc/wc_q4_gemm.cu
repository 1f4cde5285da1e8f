// wc_q4_gemm.cu -- products of 4-bit weights with many rows of activations, on
// the sm_100a tensor cores.
//
//   y[p][r] = sum_g s[r][g] * sum_{c in g} (q[r][c] - z[r][g]) * x[p][c]
//
// One thread block per SM walks units of 128 weight rows (the MMA's M) times a
// tile of up to NT rows of x (its N), swept over the columns in slices of 128.
// Roles joined by mbarrier rings, so that none waits for all the others:
//   - one thread copies each slice's records (128 rows of codes, scales and
//     zero points: one contiguous piece) into a ring in shared memory; another
//     loads the slice's activations by TMA in the 128-byte swizzled K-major
//     layout the MMA reads B in (two warps with narrower copies when the rows
//     of x are not 16-byte aligned);
//   - eight unpacking warps, four per slice in turns, one lane per row, turn
//     codes into 16-bit integers q - z and store them as the A operand into
//     tensor memory;
//   - two warps issue tcgen05.mma, each GROUP of columns into an accumulator
//     of its own in tensor memory: the products are exact and a group sums at
//     most 128 of them;
//   - sixteen scaling warps read a group's accumulator (tcgen05.ld), scale it in
//     FP32 and add it to the row's sums in registers.
// Scaling sums instead of weights keeps every weight exact (s (q - z) has up to
// 15 significant bits, a BF16 operand 8) and bounds the unspecified rounding of
// the tensor cores' accumulation to one group. Its cost is one FP32 FMA per
// result and group, beside the 1.4 instructions a weight of the unpacking.
// With few units, the blocks of a cluster share a unit's slices and add their
// sums through distributed shared memory in a fixed order: y is the same on
// every run. Every wait is bounded by the device timer.
//
// Measured (GPU time of short captured runs, BF16; beside it the larger of the bytes
// at the copy's rate and the operations at the matrix product's): 64 rows of x
// through 14336 x 4096, groups of 128, 19.4 us (5.1); 512 rows through 4096 x 14336,
// groups of 64 with zero points, 67 us (35), 0.89 PFLOP/s; 2000 rows over 8 experts
// of 14336 x 4096, groups of 128 with zero points, 258 us (137), 0.91 PFLOP/s. In
// long runs, at the power cap's clock, 77 and 310 us: 0.78 and 0.76 PFLOP/s. At 512
// rows bound by instruction issue (0.68 a cycle and scheduler, of which a third is
// useful arithmetic, the rest waits, addresses and moves around it) and, for groups
// of 64 and less, by an accumulator's round trip of some 1000 cycles (multiply,
// commit, read, hand back) with two of them; the tensor pipe is active 45 % of the
// time. At 64 rows (issue 0.39) by the latency of a slice's chain, by fetching the
// roles' instructions, and by 36 multiprocessors without a unit. Steps on
// the way (512 rows): one issuing thread, 8 + 8 warps 135 us; two issuing warps 104;
// no time limits inside polls, uniform issuing 91; one barrier a group 77; sums by
// 16 warps, pairs scaled where they were read 73; barrier addresses kept in
// registers 68.
#include <cooperative_groups.h>
#include <stddef.h>
#include <string.h>

#include "wc_q4_core.cuh"
#include "wc_ring.cuh"
#include "wc_tcgen05.cuh"

namespace wc {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t kRowsTile = 128;
constexpr uint32_t kWRing = 8;        // stages of records
constexpr uint32_t kSRing = 4;        // stages of a slice's operands: x in shared memory, A in
                                      // tensor memory
constexpr uint32_t kACol = 256;       // their first column (accumulators below)
constexpr uint32_t kAccCols = 256;
constexpr uint32_t kMaxRecBytes = kQ4Codes + 32u * 4u + 64u;
constexpr uint32_t kWStage = 8 * kMaxRecBytes;
constexpr uint32_t kSmemMax = 232448;

constexpr int kMWarps = 2;
constexpr int kWWarp = 0, kMWarp0 = 2;  // 1: activations; 2, 3: MMA issue
constexpr int kUnpWarp0 = 4;    // then the unpacking warps and the scaling warps

// Four unpacking warps a slice, slices in kUnpTurns turns; a scaling warp holds
// 32 rows' sums of up to 32 columns. Wide tiles spend their time on the sums,
// narrow ones on the codes: 16 scaling and 8 unpacking warps against 8 and 12 at
// NT = 128 measured 73 and 84 us (512 rows of x, 4096 x 14336, groups of 64), at
// NT = 64 20 and 18.5 us (64 rows, 14336 x 4096, groups of 128).
template <int NT>
struct Roles {
    static constexpr int unp_turns = NT == 128 ? 2 : 3;
    static constexpr int scl_warps = NT == 128 ? 16 : 8;
    static constexpr int scl_warp0 = kUnpWarp0 + 4 * unp_turns;
    static constexpr int warps = scl_warp0 + scl_warps;
    static constexpr int threads = 32 * warps;
    // Registers of a thread at launch and after the roles split.
    static constexpr int regs = NT == 128 ? 72 : 80;
    static constexpr int regs_issue = NT == 128 ? 48 : 64, regs_unpack = regs_issue;
    static constexpr int regs_scale = NT == 128 ? 88 : 104;
    static_assert(threads * regs <= 65536, "registers at launch");
    static_assert(4 * regs_issue + 4 * unp_turns * regs_unpack + scl_warps * regs_scale <=
                      warps * regs,
                  "the roles' registers come out of those at launch");
};

// Accumulators of NT columns: group number n of the block goes to n % accs.
template <int NT, int PER>
__host__ __device__ constexpr uint32_t accs() {
    return kAccCols / NT < kSRing * PER ? kAccCols / NT : kSRing * PER;
}

struct GmParams {
    CUtensorMap x_map;
    Q4GemmArgs a;
    Q4Layout L;
    uint32_t row_blocks;  // 128-row blocks of a matrix
    uint32_t tiles;       // one matrix: token tiles, and tokens of a tile
    uint32_t per_tile;
    uint32_t split;       // thread blocks that share a unit
    uint32_t x_bytes;     // alignment of the rows of x: 16 (TMA), 8, 4 or 2
};

struct GmCtl {
    unsigned long long w_full[kWRing], w_empty[kWRing];
    // A group's operands and a free accumulator: the one thing its issue waits
    // for. Arrivals: the unpacking warps; the scaling warps, when they have read
    // the accumulator's last group; and the activations' copy, on the first
    // group of each 64-column panel.
    unsigned long long g_full[kSRing][4];
    unsigned long long done[kSRing][4];    // the MMAs of a group
    unsigned long long s_free[kSRing];     // the MMAs of a slice (PER > 1: of both issuing warps)
    unsigned long long drain[kMWarps];
    uint32_t tmem_base;
    int abort;
};

struct GmSmem {
    GmCtl* ctl;
    uint8_t* x;
    uint8_t* w;
    uint32_t* first;   // per expert: first unit (experts + 1 values),
    uint32_t* lo;      // first row of x,
    uint32_t* cnt;     // rows
};

struct GmUnit {
    uint32_t e, tok0, ntok, rb;
    bool valid;
};

// Tiles of cnt rows: as few as NT allows, of equal sizes rounded up to 16.
template <int NT>
__device__ __forceinline__ uint32_t tile_rows(uint32_t cnt) {
    const uint32_t tiles = (cnt + NT - 1) / NT;
    return ((cnt + tiles - 1) / tiles + 15u) & ~15u;
}

// Unit u: tiles of one row block are neighbours, so that blocks running at the
// same time share its records through L2. `e` is where the search starts.
template <int NT>
__device__ __forceinline__ GmUnit unit_at(const GmParams& P, const GmSmem& S, uint32_t u,
                                          uint32_t e) {
    GmUnit t = {};
    if (P.a.offsets == nullptr) {
        t.valid = u < P.row_blocks * P.tiles;
        t.rb = u / P.tiles;
        t.tok0 = (u % P.tiles) * P.per_tile;
        t.ntok = min(P.per_tile, P.a.tokens - t.tok0);
        return t;
    }
    t.valid = u < S.first[P.a.experts];
    if (!t.valid) return t;
    while (u >= S.first[e + 1]) ++e;
    const uint32_t cnt = S.cnt[e], per = tile_rows<NT>(cnt), tiles = (cnt + per - 1) / per;
    const uint32_t k = u - S.first[e];
    t.e = e;
    t.rb = k / tiles;
    const uint32_t off = (k % tiles) * per;
    t.tok0 = S.lo[e] + off;
    t.ntok = min(per, cnt - off);
    return t;
}

// Addresses of the barriers in the shared window, from one base register that the
// compiler cannot take apart: computed from pointers, each use became a handful of
// uniform instructions, and the kernel is bound by instruction issue.
__device__ __forceinline__ uint32_t ctl_base(const GmSmem& S) {
    uint32_t a;
    asm volatile("mov.u32 %0, %1;" : "=r"(a) : "r"(smem_addr(S.ctl)));
    return a;
}
#define WC_BAR(field) (cb + uint32_t(offsetof(GmCtl, field)))

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// One poll, which suspends the thread for a while. Without a time of its own: a
// poll that names one becomes a loop of polls, sleeps and clock reads (measured
// here: 350 barrier and 160 sleep instructions a slice instead of some 75), whose
// instructions the other roles wait for.
__device__ __forceinline__ bool gm_poll(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Wait for a phase (one lane); false if another role gave up or the time limit
// passed.
__device__ __forceinline__ bool gm_wait(uint32_t bar, uint32_t parity, GmCtl& c, int32_t* status) {
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 128; ++k)
            if (gm_poll(bar, parity)) return true;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (*const_cast<volatile int*>(&c.abort)) return false;
        if (t - t0 > kWaitLimitNs) {
            report(status, kStatusTimeout);
            c.abort = 1;
            return false;
        }
    }
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 l;\n\t"
        "elect.sync l|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// The same by a whole warp, its control flow uniform throughout: the lanes' polls
// may differ, but no lane goes on before a vote, so that the warp reaches the
// warp-wide (.aligned) instructions that follow as one.
__device__ __forceinline__ bool gm_wait_warp(uint32_t bar, uint32_t parity, GmCtl& c,
                                             int32_t* status) {
    if (__builtin_expect(__all_sync(0xFFFFFFFFu, gm_poll(bar, parity)), 1)) return true;
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 128; ++k)
            if (__all_sync(0xFFFFFFFFu, gm_poll(bar, parity))) return true;
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

// A ring position: stage and how often the ring went round.
template <uint32_t N>
struct Ring {
    uint32_t s = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) s = 0, ++round;
    }
    __device__ __forceinline__ uint32_t fills() const { return round * N + s; }
    __device__ __forceinline__ uint32_t empty() const { return (round - 1u) & 1u; }
};

// The slices of a unit that this block takes.
__device__ __forceinline__ void my_slices(const GmParams& P, uint32_t& s0, uint32_t& s1) {
    const uint32_t r = blockIdx.x % P.split;
    s0 = uint32_t(uint64_t(P.L.slices) * r / P.split);
    s1 = uint32_t(uint64_t(P.L.slices) * (r + 1) / P.split);
}

// The loading roles return how many copies they started: those that may still be in
// flight when the roles end are waited for (gm_drain) if one of them gave up.
template <int NT>
__device__ uint32_t gm_load_w(const GmParams& P, const GmSmem& S) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    const Q4Layout& L = P.L;
    uint32_t s0, s1, e = 0;
    my_slices(P, s0, s1);
    Ring<kWRing> w;
    bool ok = true;
    for (uint32_t u = blockIdx.x / P.split; ok; u += gridDim.x / P.split) {
        const GmUnit t = unit_at<NT>(P, S, u, e);
        if (!t.valid) break;
        e = t.e;
        const uint8_t* stream = P.a.stream + t.e * P.a.stride;
        const uint32_t h = min(8u, L.blocks16 - 8 * t.rb);
        if (t.rb == 0 && s0 == 0) q4_check_header(stream, L, P.a.status);
        for (uint32_t s = s0; s < s1; ++s, w.next()) {
            if (w.round > 0 && !gm_wait(WC_BAR(w_empty) + 8u * (w.s), w.empty(), c, P.a.status)) {
                ok = false;
                break;
            }
            mbar_arrive_expect_tx(&c.w_full[w.s], h * L.rec);
            bulk_load(S.w + w.s * kWStage, stream + q4_record(L, 8 * t.rb, s), h * L.rec,
                      &c.w_full[w.s]);
        }
    }
    return w.fills();
}

template <int NT, int PER>
__device__ uint32_t gm_load_x_tma(const GmParams& P, const GmSmem& S) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    uint32_t s0, s1, e = 0;
    my_slices(P, s0, s1);
    Ring<kSRing> x;
    bool ok = true;
    for (uint32_t u = blockIdx.x / P.split; ok; u += gridDim.x / P.split) {
        const GmUnit t = unit_at<NT>(P, S, u, e);
        if (!t.valid) break;
        e = t.e;
        for (uint32_t s = s0; s < s1; ++s, x.next()) {
            if (x.round > 0 && !gm_wait(WC_BAR(s_free) + 8u * (x.s), x.empty(), c, P.a.status)) {
                ok = false;
                break;
            }
            uint8_t* d = S.x + x.s * NT * 256;
            unsigned long long* b0 = &c.g_full[x.s][0];
            unsigned long long* b1 = &c.g_full[x.s][PER / 2];
            mbar_arrive_expect_tx(b0, NT * (PER == 1 ? 256 : 128));
            tma_load_2d(d, &P.x_map, int32_t(s * kQ4Cols), int32_t(t.tok0), b0);
            if (PER > 1) mbar_arrive_expect_tx(b1, NT * 128);
            tma_load_2d(d + NT * 128, &P.x_map, int32_t(s * kQ4Cols + 64), int32_t(t.tok0), b1);
        }
    }
    return x.fills();
}

// No copy outlives the block: its shared memory goes to another. After an abort the
// other arrivals of a slice may never come; the first wait that runs out has given
// all copies its time.
template <int PER>
__device__ void gm_drain(GmCtl& c, uint32_t w_fills, uint32_t x_fills) {
    bool landed = true;
    ring_last_fills(w_fills, kWRing, [&](uint32_t st, uint32_t parity) {
        landed = landed && mbar_wait(&c.w_full[st], parity, nullptr);
    });
    ring_last_fills(x_fills, kSRing, [&](uint32_t st, uint32_t parity) {
        landed = landed && mbar_wait(&c.g_full[st][0], parity, nullptr) &&
                 mbar_wait(&c.g_full[st][PER / 2], parity, nullptr);
    });
}

// Rows of x that TMA cannot take: V-byte copies (V = 8, 4: cp.async; 2: through
// registers) into the same swizzled layout, zeros past the last column. A slice
// is handed over one slice later, when its copies have landed.
template <int NT, int PER, int V>
__device__ void gm_load_x_any(const GmParams& P, const GmSmem& S, uint32_t tid) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    uint32_t s0, s1, e = 0;
    my_slices(P, s0, s1);
    Ring<kSRing> x;
    int prev = -1;  // stage not yet handed over
    auto hand_over = [&](int stage) {
        fence_proxy_async_smem();
        bar_arrive(WC_BAR(g_full) + 32u * (stage) + 8u * (0));
        if (PER > 1) bar_arrive(WC_BAR(g_full) + 32u * (stage) + 8u * (PER / 2));
    };
    bool ok = true;
    for (uint32_t u = blockIdx.x / P.split; ok; u += gridDim.x / P.split) {
        const GmUnit t = unit_at<NT>(P, S, u, e);
        if (!t.valid) break;
        e = t.e;
        for (uint32_t s = s0; s < s1; ++s, x.next()) {
            if (x.round > 0 && !gm_wait_warp(WC_BAR(s_free) + 8u * (x.s), x.empty(), c, P.a.status)) {
                ok = false;
                break;
            }
            const uint32_t base = smem_addr(S.x + x.s * NT * 256);
            constexpr uint32_t W = V == 2 ? 4 : V;    // bytes a step writes
            constexpr uint32_t per_row = 256 / W;
            for (uint32_t k = tid; k < t.ntok * per_row; k += 32) {
                const uint32_t n = k / per_row, b = (k % per_row) * W;  // row, byte in the slice
                const uint32_t col = s * kQ4Cols + b / 2;
                const uint32_t bp = b & 127u;
                const uint32_t dst = base + (b >> 7) * (NT * 128) + n * 128 +
                                     ((((bp >> 4) ^ (n & 7u)) << 4) | (bp & 15u));
                const uint16_t* src =
                    static_cast<const uint16_t*>(P.a.x) + uint64_t(t.tok0 + n) * P.a.ldx + col;
                const uint32_t have = col < P.L.cols ? min(W, (P.L.cols - col) * 2) : 0u;
                if (V == 2) {
                    const uint32_t v = (have >= 2 ? uint32_t(src[0]) : 0u) |
                                       (have >= 4 ? uint32_t(src[1]) << 16 : 0u);
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
                } else {
                    const void* from = have ? static_cast<const void*>(src) : P.a.x;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst),
                                 "l"(from), "n"(V), "r"(have)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (prev >= 0) {
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                hand_over(prev);
            }
            prev = int(x.s);
        }
        if (ok && prev >= 0) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            hand_over(prev);
            prev = -1;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// Slices of all the block's units.
template <int NT>
__device__ __forceinline__ uint32_t all_slices(const GmParams& P, const GmSmem& S) {
    uint32_t s0, s1;
    my_slices(P, s0, s1);
    const uint32_t units = P.a.offsets == nullptr ? P.row_blocks * P.tiles : S.first[P.a.experts];
    const uint32_t u0 = blockIdx.x / P.split, du = gridDim.x / P.split;
    return u0 < units ? ((units - u0 + du - 1) / du) * (s1 - s0) : 0u;
}

// Unpacking warps: four a slice, the block's slices in turns.
template <int NT, bool HALF, int PER>
__device__ void gm_unpack(const GmParams& P, const GmSmem& S, int wi, int lane) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    const Q4Layout& L = P.L;
    const Q4Masks mk = Q4Masks::make<HALF>();
    const uint32_t q = uint32_t(wi) & 3u, turn = uint32_t(wi) >> 2;
    const uint32_t r = 32u * q + uint32_t(lane);
    const uint32_t row_at = smem_addr(S.w) + (r >> 4) * L.rec + (r & 15u) * 16u;
    const uint32_t zero_at = smem_addr(S.w) + (r >> 4) * L.rec + kQ4Codes + 32u * PER + (r & 15u);
    const uint32_t t_lane = ((32u * q) << 16) + kACol;
    const uint32_t total = all_slices<NT>(P, S);
    const bool zeros = L.zeros != 0;
    for (uint32_t n = turn; n < total; n += Roles<NT>::unp_turns) {
        const uint32_t ws = n % kWRing, st = n % kSRing;
        if (!gm_wait_warp(WC_BAR(w_full) + 8u * (ws), (n / kWRing) & 1u, c, P.a.status)) return;
        uint32_t zp[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            uint32_t z = 8;
            if (zeros)
                asm volatile("ld.shared.u8 %0, [%1];"
                             : "=r"(z)
                             : "r"(zero_at + ws * kWStage + 16u * k));
            zp[k] = q4_zero_pair<HALF>(z);
        }
        if (n >= kSRing &&
            !gm_wait_warp(WC_BAR(s_free) + 8u * (st), (n / kSRing - 1u) & 1u, c, P.a.status))
            return;
        tc_fence_after();
        // Stores of four registers as soon as they are there: with 16 a store the
        // warps stood still (83 against 68 us, 512 rows of x through 4096 x 14336).
        uint32_t src = row_at + ws * kWStage, dst = t_lane + st * 64u;
#pragma unroll 2
        for (int k = 0; k < 4; ++k, src += 256u, dst += 4u) {
            const uint4 v = lds128(src);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t word = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
                uint32_t o[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) o[p] = q4_pair<HALF>(word, p, zp[i * PER / 4], mk);
                tmem_st4(dst + 16u * i, o);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
            for (int g = 0; g < PER; ++g) bar_arrive(WC_BAR(g_full) + 32u * (st) + 8u * (g));
            bar_arrive(WC_BAR(w_empty) + 8u * (ws));
        }
    }
}

// MMA issue. One group a slice: the two warps take slices in turns; more: warp
// p takes the groups of the 64-column panel p of every slice. A warp's next
// wait returns only after the MMAs it issued before have left its queue (a
// barrier poll or any other read of shared memory behind 8 of them costs some
// 170 cycles), so there is one wait a group and the other warp's MMAs run
// meanwhile. The whole warp walks and one lane issues; everything an MMA is
// given is uniform to the compiler's eye (the warp's number a constant, what
// comes from shared memory through a vote or a reduction), or each operand is
// moved from a vector register in a loop of its own: 12 moves an MMA, 430
// cycles for 4 of them.
template <int NT, bool HALF, int PER, int TURN>
__device__ void gm_mma(const GmParams& P, const GmSmem& S) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    constexpr uint32_t ACCS = accs<NT, PER>();
    constexpr int kGroups = PER == 1 ? 1 : PER / 2;  // of this warp in a slice it takes
    constexpr int kMmas = 8 / PER;                   // a group
    const uint32_t x0 = smem_addr(S.x);
    uint32_t s0, s1, e = 0, count = 0;
    my_slices(P, s0, s1);
    bool ok = true, issued = false;
    for (uint32_t u = blockIdx.x / P.split; ok; u += gridDim.x / P.split) {
        const GmUnit t = unit_at<NT>(P, S, u, e);
        if (!__any_sync(0xFFFFFFFFu, t.valid)) break;
        e = t.e;
        // kind::f16: FP32 accumulator, A and B both BF16 or both FP16 (0 in bits 7-12)
        const uint32_t nn = __reduce_max_sync(0xFFFFFFFFu, (t.ntok + 15u) & ~15u);
        const uint32_t idesc = HALF ? bf16_idesc(kRowsTile, nn) & ~((1u << 7) | (1u << 10))
                                    : bf16_idesc(kRowsTile, nn);
        const uint32_t end = count + (s1 - s0);
        for (uint32_t n = PER == 1 ? count + ((count ^ TURN) & 1u) : count; ok && n < end;
             n += PER == 1 ? kMWarps : 1) {
            const uint32_t st = n % kSRing, round = n / kSRing;
            const uint32_t ta = kACol + st * 64u;
            const uint64_t xd0 = sw128_desc(x0 + st * (NT * 256));
            const uint64_t xd1 = xd0 + NT * 8;
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const uint32_t g = PER == 1 ? 0u : TURN * kGroups + j;
                if (!gm_wait_warp(WC_BAR(g_full) + 32u * (st) + 8u * (g), round & 1u, c, P.a.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = (n * PER + g) % ACCS * NT;
                // the group's first K step: 8 columns of A and 32 bytes of B each
                const uint32_t a0 = ta + 8u * kMmas * g;
                const uint64_t b0 = PER == 1 ? xd0 : (TURN ? xd1 : xd0) + 2u * kMmas * j;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kMmas; ++k)
                        umma_bf16_ts(acc, a0 + 8u * k,
                                     PER == 1 && k >= 4 ? xd1 + 2u * (k - 4) : b0 + 2u * k, idesc,
                                     k > 0 ? 1u : 0u);
                    bar_commit(WC_BAR(done) + 32u * (st) + 8u * (g));
                    if (j == kGroups - 1) bar_commit(WC_BAR(s_free) + 8u * (st));
                }
                __syncwarp();
                issued = true;
            }
        }
        count = end;
    }
    if (issued) {  // every MMA has finished before the block ends (elect.sync picks one lane
                   // throughout, so the commit covers all of the warp's)
        if (elect_one()) bar_commit(WC_BAR(drain) + 8u * (TURN));
        __syncwarp();
        // (also after a role gave up: what was issued has to end, and does)
        for (int k = 0; k < (1 << 20); ++k)
            if (__all_sync(0xFFFFFFFFu, gm_poll(WC_BAR(drain) + 8u * (TURN), 0))) break;
    }
}

// A group's results (consecutive FP32 columns of this thread's tensor memory
// lane) scaled and added to the sums, two a instruction, each FMA rounded to
// nearest; once they are read, one lane says so on `bar`. One block of assembly,
// so that the pairs stay where tcgen05.ld put them (through C++ values each
// pair was moved first).
__device__ __forceinline__ void scale_add(uint64_t (&sum)[16], uint32_t taddr, uint32_t bar,
                                          uint32_t arrive, uint64_t s2) {
    asm volatile(
        "{\n\t.reg .b32 v<32>;\n\t.reg .b64 p;\n\t.reg .pred f;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "v0,v1,v2,v3,v4,v5,v6,v7,v8,v9,v10,v11,v12,v13,v14,v15,v16,v17,v18,v19,v20,"
        "v21,v22,v23,v24,v25,v26,v27,v28,v29,v30,v31}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "tcgen05.fence::before_thread_sync;\n\t"
        "bar.warp.sync 0xFFFFFFFF;\n\t"
        "setp.ne.u32 f, %18, 0;\n\t"
        "@f mbarrier.arrive.shared::cta.b64 _, [%17];\n\t"
        "mov.b64 p, {v0, v1};\n\tfma.rn.f32x2 %0, %19, p, %0;\n\t"
        "mov.b64 p, {v2, v3};\n\tfma.rn.f32x2 %1, %19, p, %1;\n\t"
        "mov.b64 p, {v4, v5};\n\tfma.rn.f32x2 %2, %19, p, %2;\n\t"
        "mov.b64 p, {v6, v7};\n\tfma.rn.f32x2 %3, %19, p, %3;\n\t"
        "mov.b64 p, {v8, v9};\n\tfma.rn.f32x2 %4, %19, p, %4;\n\t"
        "mov.b64 p, {v10, v11};\n\tfma.rn.f32x2 %5, %19, p, %5;\n\t"
        "mov.b64 p, {v12, v13};\n\tfma.rn.f32x2 %6, %19, p, %6;\n\t"
        "mov.b64 p, {v14, v15};\n\tfma.rn.f32x2 %7, %19, p, %7;\n\t"
        "mov.b64 p, {v16, v17};\n\tfma.rn.f32x2 %8, %19, p, %8;\n\t"
        "mov.b64 p, {v18, v19};\n\tfma.rn.f32x2 %9, %19, p, %9;\n\t"
        "mov.b64 p, {v20, v21};\n\tfma.rn.f32x2 %10, %19, p, %10;\n\t"
        "mov.b64 p, {v22, v23};\n\tfma.rn.f32x2 %11, %19, p, %11;\n\t"
        "mov.b64 p, {v24, v25};\n\tfma.rn.f32x2 %12, %19, p, %12;\n\t"
        "mov.b64 p, {v26, v27};\n\tfma.rn.f32x2 %13, %19, p, %13;\n\t"
        "mov.b64 p, {v28, v29};\n\tfma.rn.f32x2 %14, %19, p, %14;\n\t"
        "mov.b64 p, {v30, v31};\n\tfma.rn.f32x2 %15, %19, p, %15;\n\t"
        "}"
        : "+l"(sum[0]), "+l"(sum[1]), "+l"(sum[2]), "+l"(sum[3]), "+l"(sum[4]),
          "+l"(sum[5]), "+l"(sum[6]), "+l"(sum[7]), "+l"(sum[8]), "+l"(sum[9]),
          "+l"(sum[10]), "+l"(sum[11]), "+l"(sum[12]), "+l"(sum[13]), "+l"(sum[14]),
          "+l"(sum[15])
        : "r"(taddr), "r"(bar), "r"(arrive), "l"(s2)
        : "memory");
}

__device__ __forceinline__ void scale_add(uint64_t (&sum)[8], uint32_t taddr, uint32_t bar,
                                          uint32_t arrive, uint64_t s2) {
    asm volatile(
        "{\n\t.reg .b32 v<16>;\n\t.reg .b64 p;\n\t.reg .pred f;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "v0,v1,v2,v3,v4,v5,v6,v7,v8,v9,v10,v11,v12,v13,v14,v15}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "tcgen05.fence::before_thread_sync;\n\t"
        "bar.warp.sync 0xFFFFFFFF;\n\t"
        "setp.ne.u32 f, %10, 0;\n\t"
        "@f mbarrier.arrive.shared::cta.b64 _, [%9];\n\t"
        "mov.b64 p, {v0, v1};\n\tfma.rn.f32x2 %0, %11, p, %0;\n\t"
        "mov.b64 p, {v2, v3};\n\tfma.rn.f32x2 %1, %11, p, %1;\n\t"
        "mov.b64 p, {v4, v5};\n\tfma.rn.f32x2 %2, %11, p, %2;\n\t"
        "mov.b64 p, {v6, v7};\n\tfma.rn.f32x2 %3, %11, p, %3;\n\t"
        "mov.b64 p, {v8, v9};\n\tfma.rn.f32x2 %4, %11, p, %4;\n\t"
        "mov.b64 p, {v10, v11};\n\tfma.rn.f32x2 %5, %11, p, %5;\n\t"
        "mov.b64 p, {v12, v13};\n\tfma.rn.f32x2 %6, %11, p, %6;\n\t"
        "mov.b64 p, {v14, v15};\n\tfma.rn.f32x2 %7, %11, p, %7;\n\t"
        "}"
        : "+l"(sum[0]), "+l"(sum[1]), "+l"(sum[2]), "+l"(sum[3]), "+l"(sum[4]),
          "+l"(sum[5]), "+l"(sum[6]), "+l"(sum[7])
        : "r"(taddr), "r"(bar), "r"(arrive), "l"(s2)
        : "memory");
}

__device__ __forceinline__ uint64_t pair2(float s) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(s));
    return d;
}
__device__ __forceinline__ float half2f(uint64_t v, int hi) {
    return __uint_as_float(uint32_t(hi ? v >> 32 : v));
}

template <int NT, bool HALF, int PER>
__device__ void gm_scale(const GmParams& P, const GmSmem& S, int wi, int lane) {
    GmCtl& c = *S.ctl;
    const uint32_t cb = ctl_base(S);
    const Q4Layout& L = P.L;
    constexpr uint32_t ACCS = accs<NT, PER>();
    constexpr int HN = NT / (Roles<NT>::scl_warps / 4);  // columns of this warp
    const uint32_t q = uint32_t(wi) & 3u, part = uint32_t(wi) >> 2;
    const uint32_t r = 32u * q + uint32_t(lane);
    const uint32_t scale_at = smem_addr(S.w) + (r >> 4) * L.rec + kQ4Codes + (r & 15u) * 2u;
    const uint32_t half_scales = L.half_scales;
    const uint32_t t_lane = ((32u * q) << 16) + part * HN;
    uint32_t s0, s1, e = 0, count = 0;
    my_slices(P, s0, s1);
    if (lane == 0)  // the first groups' accumulators are free
        for (uint32_t k = 0; k < ACCS; ++k) bar_arrive(WC_BAR(g_full) + 32u * (k / PER) + 8u * (k % PER));
    for (uint32_t u = blockIdx.x / P.split;; u += gridDim.x / P.split) {
        const GmUnit t = unit_at<NT>(P, S, u, e);
        if (!t.valid) return;
        e = t.e;
        uint64_t sum[HN / 2];
#pragma unroll
        for (int k = 0; k < HN / 2; ++k) sum[k] = 0;  // two FP32 zeros
        const uint32_t live = t.ntok > part * HN ? t.ntok - part * HN : 0u;  // columns in use
        for (const uint32_t end = count + (s1 - s0); count < end; ++count) {
            const uint32_t st = count % kSRing, round = count / kSRing, ws = count % kWRing;
#pragma unroll
            for (int g = 0; g < PER; ++g) {
                const uint32_t gi = count * PER + g, next = gi + ACCS;
                if (!gm_wait_warp(WC_BAR(done) + 32u * (st) + 8u * (g), round & 1u, c, P.a.status)) return;
                tc_fence_after();
                // The group's MMAs are done, so its records have long landed
                // (the unpacking warps waited for them) and stay until this
                // warp's word on w_empty: no wait of its own.
                uint16_t bits;
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(bits)
                             : "r"(scale_at + ws * kWStage + 32u * g));
                const uint64_t sc = pair2(q4_scale(bits, half_scales));
                const uint32_t bar =
                    WC_BAR(g_full) + 32u * (next / PER % kSRing) + 8u * (next % PER);
                if (live > 0) {
                    scale_add(sum, t_lane + gi % ACCS * NT, bar, lane == 0, sc);
                } else {
                    if (lane == 0) bar_arrive(bar);
                }
                if (g == PER - 1) {
                    __syncwarp();
                    if (lane == 0) bar_arrive(WC_BAR(w_empty) + 8u * (ws));
                }
            }
        }
        if (P.split == 1) {
            const uint32_t row = t.rb * kRowsTile + r;
            if (row < L.rows) {
#pragma unroll
                for (int k = 0; k < HN; ++k)
                    if (uint32_t(k) < live)
                        q4_store<HALF>(P.a, uint64_t(t.tok0) + part * HN + k, row,
                                      half2f(sum[k / 2], k & 1));
            }
        } else {  // the block's only unit: every copy into the ring has been used
            float* red = reinterpret_cast<float*>(S.x);
#pragma unroll
            for (int k = 0; k < HN; ++k)
                red[(part * HN + k) * kRowsTile + r] = half2f(sum[k / 2], k & 1);
        }
    }
}

template <int NT, bool HALF, int PER>
__global__ void __launch_bounds__(Roles<NT>::threads, 1)
    q4_gemm_kernel(const __grid_constant__ GmParams P) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // uniform
    uint8_t* p = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    GmSmem S;
    S.x = p;
    p += kSRing * NT * 256;
    S.w = p;
    p += kWRing * kWStage;
    S.ctl = reinterpret_cast<GmCtl*>(p);
    p += (sizeof(GmCtl) + 15) / 16 * 16;
    S.first = reinterpret_cast<uint32_t*>(p);
    S.lo = S.first + P.a.experts + 1;
    S.cnt = S.lo + P.a.experts;
    GmCtl& c = *S.ctl;
    if (tid == 0) {
        for (uint32_t s = 0; s < kWRing; ++s) {
            mbar_init(&c.w_full[s], 1);
            mbar_init(&c.w_empty[s], 4 + Roles<NT>::scl_warps);
        }
        for (uint32_t s = 0; s < kSRing; ++s) {
            for (int g = 0; g < PER; ++g) {
                const bool first = g == 0 || (PER > 1 && g == PER / 2);  // of a panel
                mbar_init(&c.g_full[s][g],
                          4 + Roles<NT>::scl_warps + (!first ? 0 : P.x_bytes == 16 ? 1 : 32));
                mbar_init(&c.done[s][g], 1);
            }
            mbar_init(&c.s_free[s], PER == 1 ? 1 : kMWarps);
        }
        for (int s = 0; s < kMWarps; ++s) mbar_init(&c.drain[s], 1);
        c.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMWarp0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&c.tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (P.a.offsets != nullptr) {  // the experts' rows and first units
        const int total = int(P.a.tokens);
        for (uint32_t e = tid; e < P.a.experts; e += Roles<NT>::threads) {
            const int lo = min(max(P.a.offsets[e], 0), total);
            const int hi = min(max(P.a.offsets[e + 1], lo), total);
            const uint32_t cnt = uint32_t(hi - lo);
            S.lo[e] = uint32_t(lo);
            S.cnt[e] = cnt;
            const uint32_t per = cnt ? tile_rows<NT>(cnt) : 1u;
            S.first[e + 1] = (cnt + per - 1) / per * P.row_blocks;
        }
        __syncthreads();
        if (warp == 0) {
            uint32_t run = 0;
            for (uint32_t e0 = 0; e0 < P.a.experts; e0 += 32) {
                const uint32_t e = e0 + lane;
                uint32_t v = e < P.a.experts ? S.first[e + 1] : 0u;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, v, o);
                    if (lane >= o) v += x;
                }
                if (e < P.a.experts) S.first[e + 1] = run + v;
                run += __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (lane == 0) S.first[0] = 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All 512 columns are this block's, so its tensor memory starts at address 0,
    // which the roles use as a constant (and do nothing, were it ever otherwise).
    const bool run = c.tmem_base == 0;
    if (!run && tid == 0) {
        report(P.a.status, kStatusTimeout);
        c.abort = 1;
    }

    if (warp < kUnpWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs_issue));
        uint32_t w_fills = 0, x_fills = 0;
        if (warp == kWWarp) {
            if (lane == 0 && run) w_fills = gm_load_w<NT>(P, S);
        } else if (!run) {
        } else if (warp >= kMWarp0) {
            if (warp == kMWarp0)
                gm_mma<NT, HALF, PER, 0>(P, S);
            else
                gm_mma<NT, HALF, PER, 1>(P, S);
        } else if (P.x_bytes == 16) {
            if (lane == 0) x_fills = gm_load_x_tma<NT, PER>(P, S);
        } else if (P.x_bytes == 8) {
            gm_load_x_any<NT, PER, 8>(P, S, lane);
        } else if (P.x_bytes == 4) {
            gm_load_x_any<NT, PER, 4>(P, S, lane);
        } else {
            gm_load_x_any<NT, PER, 2>(P, S, lane);
        }
        __syncwarp();     // (of roles that one lane takes)
        __syncthreads();  // (no warp spins for the registers that the scaling warps hold)
        if (w_fills + x_fills > 0 && c.abort) gm_drain<PER>(c, w_fills, x_fills);
        __syncwarp();
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs));
    } else if (warp < Roles<NT>::scl_warp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs_unpack));
        if (run) gm_unpack<NT, HALF, PER>(P, S, warp - kUnpWarp0, lane);
        __syncthreads();
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs));
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs_scale));
        if (run) gm_scale<NT, HALF, PER>(P, S, warp - Roles<NT>::scl_warp0, lane);
        __syncthreads();
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<NT>::regs));
    }
    __syncwarp();
    if (P.split > 1) {
        if (c.abort) {  // (the roles have ended: the same for all threads)
            __syncthreads();  // the last copies into this memory have landed
            float* red = reinterpret_cast<float*>(S.x);
            for (uint32_t k = tid; k < NT * kRowsTile; k += Roles<NT>::threads)
                red[k] = __int_as_float(0x7FC00000);  // no sums: the results are NaN
        }
        // each block of the cluster adds and writes its share of the tokens
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const GmUnit t = unit_at<NT>(P, S, blockIdx.x / P.split, 0);
        if (t.valid) {
            const uint32_t rank = blockIdx.x % P.split;
            const float* red = reinterpret_cast<const float*>(S.x);
            const uint32_t t0 = t.ntok * rank / P.split, t1 = t.ntok * (rank + 1) / P.split;
            for (uint32_t k = t0 * kRowsTile + tid; k < t1 * kRowsTile; k += Roles<NT>::threads) {
                float v = 0.f;
                for (uint32_t b = 0; b < P.split; ++b) v += cluster.map_shared_rank(red, b)[k];
                const uint32_t row = t.rb * kRowsTile + k % kRowsTile;
                if (row < P.L.rows) q4_store<HALF>(P.a, uint64_t(t.tok0) + k / kRowsTile, row, v);
            }
        }
        cluster.sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMWarp0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.tmem_base),
                     "r"(512)
                     : "memory");
    }
}

template <int NT>
uint32_t gm_smem(uint32_t experts) {
    return 1024 + kSRing * NT * 256 + kWRing * kWStage + (sizeof(GmCtl) + 15) / 16 * 16 +
           (3 * experts + 1) * 4;
}

template <int NT, bool HALF, int PER>
cudaError_t gm_launch(GmParams& P, uint32_t sms, uint32_t units, cudaStream_t stream) {
    static std::mutex mu;
    static bool set[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = q4_gemm_kernel<NT, HALF, PER>;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(kSmemMax));
            if (err != cudaSuccess) return err;
            set[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(P.split > 1 ? units * P.split : units < sms ? units : sms);
    cfg.blockDim = dim3(Roles<NT>::threads);
    cfg.dynamicSmemBytes = gm_smem<NT>(P.a.experts);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = P.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <int NT>
cudaError_t gm_tokens(GmParams& P, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    P.row_blocks = (P.L.blocks16 + 7) / 8;
    const uint32_t T = P.a.tokens;
    uint64_t units;
    if (P.a.offsets == nullptr) {
        const uint32_t tiles = (T + NT - 1) / NT;
        P.per_tile = ((T + tiles - 1) / tiles + 15u) & ~15u;
        P.tiles = (T + P.per_tile - 1) / P.per_tile;
        units = uint64_t(P.row_blocks) * P.tiles;
    } else {  // at most: every expert with rows ends in a partial tile
        units = uint64_t(P.row_blocks) * (T / NT + (T < P.a.experts ? T : P.a.experts));
    }
    if (units > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    P.split = 1;
    if (P.a.offsets == nullptr)
        while (P.split < 8 && units * P.split * 2 <= uint64_t(sms) && P.L.slices / (2 * P.split) >= 4)
            P.split *= 2;
    if (P.x_bytes == 16) {
        PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
        if (enc == nullptr) return cudaErrorNotSupported;
        const bool half = P.a.flags & kQ4XHalf;
        const cuuint64_t dims[2] = {P.L.cols, T};
        const cuuint64_t strides[1] = {P.a.ldx * 2};
        const cuuint32_t box[2] = {64, NT};
        const cuuint32_t estr[2] = {1, 1};
        if (enc(&P.x_map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                const_cast<void*>(P.a.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const uint32_t u = uint32_t(units), n = uint32_t(sms);
    if (P.a.flags & kQ4XHalf)
        return P.L.per == 1   ? gm_launch<NT, true, 1>(P, n, u, stream)
               : P.L.per == 2 ? gm_launch<NT, true, 2>(P, n, u, stream)
                              : gm_launch<NT, true, 4>(P, n, u, stream);
    return P.L.per == 1   ? gm_launch<NT, false, 1>(P, n, u, stream)
           : P.L.per == 2 ? gm_launch<NT, false, 2>(P, n, u, stream)
                          : gm_launch<NT, false, 4>(P, n, u, stream);
}

}  // namespace

cudaError_t launch_q4_gemm(const Q4GemmArgs& a, const Q4Layout& L, cudaStream_t stream) {
    if (L.rows == 0 || a.tokens == 0) return cudaSuccess;
    GmParams P;
    memset(&P, 0, sizeof(P));
    P.a = a;
    P.L = L;
    // a tensor map wants 16-byte rows and at most 2^40 bytes between them
    const uint64_t al = reinterpret_cast<uintptr_t>(a.x) | (a.ldx * 2);
    P.x_bytes = al % 16 == 0 && a.ldx < (1ull << 38) ? 16u : al % 8 == 0 ? 8u : al % 4 == 0 ? 4u : 2u;
    // rows of x that a matrix takes: the tile's size follows
    const uint32_t rows = a.offsets == nullptr ? a.tokens : (a.tokens + a.experts - 1) / a.experts;
    if (rows > 64) return gm_tokens<128>(P, stream);
    if (rows > 32) return gm_tokens<64>(P, stream);
    return gm_tokens<32>(P, stream);
}

}  // namespace wc
