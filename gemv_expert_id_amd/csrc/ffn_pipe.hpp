// Pipelined products of the feed-forward block: 16-byte aligned rows whose length
// is a multiple of 16 bytes. Operands go from memory straight into LDS
// (buffer_load ... lds, 1 KiB an instruction), several stages ahead of the matrix
// instructions that read them.
//
// Reads past an operand's rows, or past a row's last chunk, carry an offset beyond
// the buffer resource's range: they give zeros without a memory access. Every loop
// therefore issues the same loads in every round, the last ones included, and each
// wait counts the same number of loads in flight.
#pragma once

#include <type_traits>
#include <utility>

#include "ffn_tile.hpp"

namespace mmk {

constexpr uint32_t kPastEnd = 0x80000000u;  // beyond every resource's range

template <int... I, class F>
__device__ __forceinline__ void ffn_for(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void ffn_for(F&& f) {
    ffn_for(std::make_integer_sequence<int, N>{}, f);
}

// s_waitcnt immediate: vmcnt <= n, lgkmcnt <= 0, expcnt untouched.
constexpr int ffn_wait(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int64_t first, int64_t ld,
                                                            int64_t rows, int64_t bytes) {
    const char* p = static_cast<const char*>(base) + first * ld;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0,
                                             rows > 0 ? (int)((rows - 1) * ld + bytes) : 0, 0x00020000);
}

#define MM_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// ---------------------------------------------------------------------------
// Few tokens: 16 FM tokens by 16 rows of W, the contraction in stages of 256 bytes.
//
// Bound by memory. W is read once, 256 contiguous bytes of a row at a time, and the tokens' pieces
// with it (from L2). A stage is four steps of matrix instructions, one for each
// wave; the waves' sums are joined through LDS at the end. So narrow a tile keeps
// many blocks in flight: one token through 22016 x 4096 takes 35.1 us in f16 (5.1
// TB/s), 41.6 with 64 rows a block and unsplit steps; through 1024 x 8192, 10.3 and
// 16.9. Chunk c of LDS row r lies at slot c ^ (r & 15), so the 16 rows of a fragment
// read cover all banks.
//
// Gated, a fragment's 16 rows are eight of the gate and the same eight of the up
// projection: the two sums of an output end 32 lanes apart.
// ---------------------------------------------------------------------------
constexpr int TStage = 256;  // bytes of k a stage
constexpr int TRows = 16;    // rows of W
constexpr int TWaves = 4;    // one for each 64-byte step of a stage

template <int FM>
struct ThinShape {
    static constexpr int XR = 16 * FM;    // tokens
    static constexpr int LOADS = FM + 1;  // of a wave and stage
    static constexpr int BYTES = (XR + TRows) * TStage;
};

// Stage S of the ring: arrays of their own, so that the compiler sees that reads of
// one stage do not meet the loads in flight into others.
template <int BYTES, int S>
__device__ __forceinline__ char* thin_stage() {
    __shared__ __attribute__((aligned(1024))) char st[BYTES];
    return st;
}

// RING stages in LDS.
template <class Out, int FM, int RING>
__global__ __launch_bounds__(64 * TWaves) void ffn_thin(FfnArgs a, int tiles_m) {
    using E = typename Out::E;
    using Acc = typename AccOf<E>::type;
    using Z = ThinShape<FM>;
    constexpr bool G = Out::kGated;
    constexpr int WO = G ? TRows / 2 : TRows;  // outputs
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lq = lane >> 4;
    // Token tiles of the same rows of W follow each other on one XCD.
    const int64_t tiles = (int64_t)tiles_m * ((a.n + WO - 1) / WO);
    const int64_t per_xcd = (tiles + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    if (t >= tiles) return;
    const int64_t m0 = t % tiles_m * Z::XR, n0 = t / tiles_m * WO;
    const int64_t bytes = a.k * (int64_t)sizeof(typename E::store_t);
    const int chunks = (int)(bytes / 16), stages = (int)((bytes + TStage - 1) / TStage);
    const int ldx = (int)a.ldx, ldw = (int)a.ldw;
    const int64_t xrows = a.m - m0 < Z::XR ? a.m - m0 : Z::XR, wrows = a.n - n0 < WO ? a.n - n0 : WO;
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, m0, a.ldx, xrows, bytes);
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w, n0, a.ldw, wrows, bytes);
    const __amdgpu_buffer_rsrc_t ru = rows_rsrc(a.w, n0 + (G ? a.n : 0), a.ldw, wrows, bytes);

    // A load covers four LDS rows; the lane fetches the chunk that belongs at slot
    // lane % 16 of row lane / 16.
    const int c0 = (lane & 15) ^ (lane >> 4), r4 = lane >> 4;
    auto issue = [&](auto S_, int st) {
        char* base = thin_stage<Z::BYTES, decltype(S_)::value>();
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int row = (w * FM + j) * 4, c = c0 ^ (row & 12);
            const uint32_t at = st * 16 + c < chunks ? (uint32_t)(r4 * ldx + c * 16) : kPastEnd;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MM_LDS(base + row * TStage), 16, at,
                                                     row * ldx + st * TStage, 0, 0);
        }
        const int row = w * 4, c = c0 ^ row;
        const uint32_t at = st * 16 + c < chunks ? (uint32_t)(r4 * ldw + c * 16) : kPastEnd;
        const bool up = G && w >= 2;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ru : rw, MM_LDS(base + (Z::XR + row) * TStage), 16, at,
                                                 (G ? row & 7 : row) * ldw + st * TStage, 0, 0);
    };
    // f32 sums run in four chains, one for each component of the lanes' chunks.
    constexpr int CH = E::code == 0 ? 4 : 1;
    Acc chain[FM][CH];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 0; q < CH; ++q) chain[i][q] = Acc{0, 0, 0, 0};
    auto compute = [&](auto S_) {
        const char* base = thin_stage<Z::BYTES, decltype(S_)::value>();
        const int at = ((4 * w + lq) ^ lr) * 16;
        const u32x4 wf = *reinterpret_cast<const u32x4*>(base + (Z::XR + lr) * TStage + at);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const u32x4 xf = *reinterpret_cast<const u32x4*>(base + (i * 16 + lr) * TStage + at);
            if constexpr (E::code == 0) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    chain[i][q] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        __uint_as_float(wf[q]), __uint_as_float(xf[q]), chain[i][q], 0, 0, 0);
            } else {
                chain[i][0] = step_mma<E>(wf, xf, chain[i][0]);
            }
        }
    };
    ffn_for<RING - 1>([&](auto S_) { issue(S_, decltype(S_)::value); });
    for (int st = 0; st < stages; st += RING) {
        ffn_for<RING>([&](auto S_) {
            constexpr int s = decltype(S_)::value;
            // Stage st + s has landed; the stage before it has been read by every wave.
            __builtin_amdgcn_s_waitcnt(ffn_wait((RING - 2) * Z::LOADS));
            __builtin_amdgcn_s_barrier();
            issue(std::integral_constant<int, (s + RING - 1) % RING>{}, st + s + RING - 1);
            compute(S_);
        });
    }
    __builtin_amdgcn_s_waitcnt(ffn_wait(0));  // no load into LDS outlives its wave
    Acc acc[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        acc[i] = chain[i][0];
        if constexpr (E::code == 0) acc[i] = (acc[i] + chain[i][1]) + (chain[i][2] + chain[i][3]);
    }
    __syncthreads();
    Acc* part = reinterpret_cast<Acc*>(thin_stage<Z::BYTES, 0>());
    static_assert((TWaves - 1) * FM * 64 * 16 <= Z::BYTES, "partial sums fit a stage");
    if (w > 0) {
#pragma unroll
        for (int i = 0; i < FM; ++i) part[((w - 1) * FM + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int q = 1; q < TWaves; ++q) acc[i] += part[((q - 1) * FM + i) * 64 + lane];
    const Out out{a};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row = m0 + i * 16 + lr;
        if constexpr (G) {
            Acc u;
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] = __shfl_xor(acc[i][q], 32, kWave);
            if (lq < 2 && row < a.m) out.pair(row, n0 + 4 * lq, acc[i], u);
        } else {
            if (row < a.m) out.one(row, n0 + 4 * lq, acc[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: WM x WN waves of 16 FM tokens x 16 FN rows of W each, the
// contraction in pairs of 64-byte steps.
//
// A region of LDS holds 128 bytes of every row of a tile (chunk c of row r at slot
// c ^ (r & 7)); a load covers 8 rows. Of a pair's two steps, the second's barrier
// frees its region for the pair NREG later, whose loads go out between the matrix
// instructions of the next two half steps. Gated, a wave's rows of W are half gate,
// half up projection, so an output's two sums end in one lane.
//
// The largest tile, 8 waves of 128 x 64, is bound by LDS and power together: a pair is
// 2048 cycles of matrix instructions and, at 128 bytes a cycle, 1536 of fragment reads
// and 512 of loads, at 1750 to 2050 MHz under this load. 8192 x 8192 over 8192: 808 us in
// bf16 (1360 TFLOP/s), 466 in codes (2360 TOP/s). Few tiles are bound by memory: 48 tokens
// by 22016 x 4096 bf16 take 41.4 us, 4.4 TB/s.
//
// XK, WK = false (16-bit gradients' products): the operand is stored with the
// contraction along its rows, element (i, p) at p * ld + i. Its region holds the
// pair's 64 k-rows of BM (BN) elements (chunk c of k-row r at slot c ^ k_swizzle(r)),
// fragments take two transposing reads, and the resource moves on with the pair, so
// that no offset grows with the contraction; k-rows past the end lie outside it.
// ---------------------------------------------------------------------------
template <int WM_, int WN_, int FM_, int FN_, int NREG_>
struct PipeShape {
    static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_, NREG = NREG_;
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN;   // tile: tokens, rows of W
    static constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES;  // loads of a wave and pair
    static_assert(XI * 8 * WAVES == BM && WI * 8 * WAVES == BN, "whole loads");
    static constexpr int LOADS = XI + WI, HALF = LOADS / 2;      // sent out in two halves
    static constexpr int REGION = (BM + BN) * 128;
    static constexpr size_t LDS = (size_t)NREG * REGION;
    static constexpr int BLOCKS = 160 * 1024 / LDS >= 2 ? 2 : 1;  // of a CU, at least
};

constexpr int PipeGroup = 4;  // tile-rows of a group: neighbours in time share W through L2

__device__ __forceinline__ int k_swizzle(int r) { return 2 * ((r & 3) + 4 * ((r >> 3) & 1)); }

// Region R of operand OP where one is strided: arrays of their own, so that the
// compiler sees that transposing reads of one do not meet loads into the others.
template <int BYTES, int R, int OP>
__device__ __forceinline__ char* pipe_region() {
    __shared__ __attribute__((aligned(1024))) char st[BYTES];
    return st;
}

extern __shared__ __attribute__((aligned(1024))) char pipe_lds[];  // (where both operands are contiguous)

// One tile: tokens from m0 on, outputs from n0 on.
template <class Out, class Z, bool XK, bool WK>
__device__ __forceinline__ void pipe_tile(const FfnArgs& a, int64_t m0, int64_t n0) {
    using E = typename Out::E;
    using Acc = typename AccOf<E>::type;
    constexpr bool G = Out::kGated;
    constexpr int BM = Z::BM, BN = Z::BN, FM = Z::FM, FN = Z::FN, HF = FM / 2, NREG = Z::NREG;
    constexpr int TM = 16 * FM, TN = 16 * FN;        // wave tile
    constexpr int WO = G ? BN / 2 : BN;              // outputs of a tile
    constexpr int LPP = Z::LOADS, LA = Z::HALF, LB = LPP - LA;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / Z::WN, wn = w % Z::WN, lr = lane & 15, lq = lane >> 4;

    constexpr bool SPLIT = !XK || !WK;  // regions as arrays of their own
    static_assert(!SPLIT || (!G && sizeof(typename E::store_t) == 2 && BM >= 128 && BN >= 128), "strided operands");
    const int64_t bytes = a.k * (int64_t)sizeof(typename E::store_t);
    const int chunks = (int)((bytes + 15) / 16);  // (whole ones where an operand is contiguous)
    const int pairs = ((chunks + 7) / 8 + NREG - 1) / NREG * NREG;
    const int ldx = (int)a.ldx, ldw = (int)a.ldw;
    const int64_t xrows = a.m - m0 < BM ? a.m - m0 : BM, wrows = a.n - n0 < WO ? a.n - n0 : WO;
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, XK ? m0 : 0, a.ldx, XK ? xrows : 0, bytes);
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w, WK ? n0 : 0, a.ldw, WK ? wrows : 0, bytes);
    const __amdgpu_buffer_rsrc_t ru = rows_rsrc(a.w, WK ? n0 + (G ? a.n : 0) : 0, a.ldw, WK ? wrows : 0, bytes);
    // Strided: the k-rows of pair p, `rows` elements of each from `first` on. (A dword
    // of the last one that reaches past them holds one of them: it is inside.)
    auto pair_rsrc = [&](const void* base, int64_t first, int64_t ld, int64_t rows, int p) {
        const int64_t left = a.k - (int64_t)p * 64, k_rows = left < 64 ? left : 64;
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(static_cast<const char*>(base) + (left > 0 ? (int64_t)p * 64 * ld : 0) + first * 2), (short)0,
            left > 0 ? (int)((k_rows - 1) * ld + (rows * 2 + 3) / 4 * 4) : 0, 0x00020000);
    };
    // Contiguous: a load covers 8 rows, the lane the chunk that belongs at slot lane % 8.
    const int dch = (lane & 7) ^ (lane >> 3);
    const int vox = (lane >> 3) * ldx + dch * 16, vow = (lane >> 3) * ldw + dch * 16;
    // Strided: a load covers 512 / B k-rows of B elements.
    constexpr int XC = BM / 8, WC = BN / 8;  // chunks of a k-row
    int vkx[XK ? 1 : Z::XI], vkw[WK ? 1 : Z::WI];
    if constexpr (!XK) {
#pragma unroll
        for (int q = 0; q < Z::XI; ++q)
            vkx[q] = lane / XC * ldx + (lane % XC ^ k_swizzle((w * Z::XI + q) * (64 / XC) + lane / XC)) * 16;
    }
    if constexpr (!WK) {
#pragma unroll
        for (int q = 0; q < Z::WI; ++q)
            vkw[q] = lane / WC * ldw + (lane % WC ^ k_swizzle((w * Z::WI + q) * (64 / WC) + lane / WC)) * 16;
    }
    auto region_x = [&](auto R_) -> char* {
        if constexpr (SPLIT) return pipe_region<BM * 128, decltype(R_)::value, 0>();
        else return pipe_lds + decltype(R_)::value * Z::REGION;
    };
    auto region_w = [&](auto R_) -> char* {
        if constexpr (SPLIT) return pipe_region<BN * 128, decltype(R_)::value, 1>();
        else return pipe_lds + decltype(R_)::value * Z::REGION + BM * 128;
    };

    // Load q of pair p into region R: x first, then W.
    auto dma = [&](auto R_, int p, auto Q_) {
        constexpr int q = decltype(Q_)::value;
        const bool live = p * 8 + dch < chunks;
        if constexpr (q < Z::XI) {
            const int i = w * Z::XI + q;
            if constexpr (XK) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MM_LDS(region_x(R_) + i * 1024), 16,
                                                         live ? (uint32_t)vox : kPastEnd, i * 8 * ldx + p * 128, 0, 0);
            } else {
                const __amdgpu_buffer_rsrc_t rp = pair_rsrc(a.x, m0, a.ldx, xrows, p);
                const int at = vkx[q];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, MM_LDS(region_x(R_) + i * 1024), 16, at,
                                                         i * (64 / XC) * ldx, 0, 0);
            }
        } else {
            const int i = w * Z::WI + q - Z::XI, row = i * 8;
            const bool up = G && row % TN >= TN / 2;
            const int col = G ? row / TN * (TN / 2) + row % (TN / 2) : row;
            if constexpr (WK) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ru : rw, MM_LDS(region_w(R_) + i * 1024), 16,
                                                         live ? (uint32_t)vow : kPastEnd, col * ldw + p * 128, 0, 0);
            } else {
                const __amdgpu_buffer_rsrc_t rp = pair_rsrc(a.w, n0, a.ldw, wrows, p);
                const int at = vkw[q - Z::XI];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, MM_LDS(region_w(R_) + i * 1024), 16, at,
                                                         i * (64 / WC) * ldw, 0, 0);
            }
        }
    };
    Acc acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    const int f0 = lr * 128 + ((lq ^ (lr & 7)) << 4), f1 = lr * 128 + (((4 + lq) ^ (lr & 7)) << 4);
    // Strided: lane s of group g addresses k-rows 8 g + s / 4 and + 4 of the step, columns
    // 4 (s % 4) on; a fragment's columns are an exclusive or away.
    const int kr = 8 * lq + (lr >> 2), kc = ((((lr & 3) >> 1) ^ k_swizzle(kr)) << 4) + 8 * (lr & 1);
    auto strided = [&](const char* region, int h, int row0, int b) {
        const char* at = region + (h * 32 + kr) * 2 * b + (kc ^ (row0 * 2));
        const u32x2 lo = read_transposed(at), hi = read_transposed(at + 8 * b);
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    // Step S (region S / 2, half S % 2): x fragments of half hh of the wave's rows, all of W's.
    auto rdx = [&](auto S_, int hh, u32x4 (&f)[HF]) {
        constexpr int s = decltype(S_)::value;
        const char* p = region_x(std::integral_constant<int, s / 2>{});
        const int row0 = wm * TM + hh * (TM / 2);
#pragma unroll
        for (int i = 0; i < HF; ++i) {
            if constexpr (XK) f[i] = *reinterpret_cast<const u32x4*>(p + (row0 + i * 16) * 128 + (s % 2 ? f1 : f0));
            else f[i] = strided(p, s % 2, row0 + i * 16, BM);
        }
    };
    auto rdw = [&](auto S_, u32x4 (&f)[FN]) {
        constexpr int s = decltype(S_)::value;
        const char* p = region_w(std::integral_constant<int, s / 2>{});
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            if constexpr (WK) f[j] = *reinterpret_cast<const u32x4*>(p + (wn * TN + j * 16) * 128 + (s % 2 ? f1 : f0));
            else f[j] = strided(p, s % 2, wn * TN + j * 16, BN);
        }
    };
    constexpr int RX = XK ? HF : 2 * HF, RW = WK ? FN : 2 * FN;  // LDS reads of each
    auto mma = [&](int hh, const u32x4 (&fx)[HF], const u32x4 (&fw)[FN]) {
#pragma unroll
        for (int i = 0; i < HF; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[hh * HF + i][j] = step_mma<E>(fw[j], fx[i], acc[hh * HF + i][j]);
    };
    // Fragment reads first, then the loads spread over the matrix instructions.
    auto weave = [&](auto READS, auto LOADS_) {
        constexpr int n = decltype(LOADS_)::value, all = HF * FN;
        __builtin_amdgcn_sched_group_barrier(0x100, decltype(READS)::value, 0);
        ffn_for<(n > 0 ? n : 1)>([&](auto Q_) {
            constexpr int q = decltype(Q_)::value, d = n > 0 ? n : 1;
            __builtin_amdgcn_sched_group_barrier(0x008, all * (q + 1) / d - all * q / d, 0);
            if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        });
        __builtin_amdgcn_sched_barrier(0);
    };
    u32x4 x0[HF], x1[HF], w0[FN], w1[FN];
    // Both steps of pair p, in region R. The first half of step 0 sends out the
    // rest of pair p + NREG - 1, the second half of step 1 the first loads of
    // pair p + NREG.
    auto pair = [&](auto R_, int p) {
        constexpr int R = decltype(R_)::value, RP = (R + NREG - 1) % NREG, RN = (R + 1) % NREG;
        using S0 = std::integral_constant<int, 2 * R>;
        using S1 = std::integral_constant<int, 2 * R + 1>;
        using SN = std::integral_constant<int, 2 * RN>;
        rdx(S0{}, 1, x1);
        ffn_for<LB>([&](auto Q_) {
            dma(std::integral_constant<int, RP>{}, p + NREG - 1, std::integral_constant<int, LA + decltype(Q_)::value>{});
        });
        mma(0, x0, w0);
        weave(std::integral_constant<int, RX>{}, std::integral_constant<int, LB>{});
        rdx(S1{}, 0, x0);
        rdw(S1{}, w1);
        mma(1, x1, w0);
        weave(std::integral_constant<int, RX + RW>{}, std::integral_constant<int, 0>{});
        rdx(S1{}, 1, x1);
        mma(0, x0, w1);
        weave(std::integral_constant<int, RX>{}, std::integral_constant<int, 0>{});
        __builtin_amdgcn_s_waitcnt(ffn_wait((NREG - 2) * LPP));  // pair p + 1 has landed
        __builtin_amdgcn_s_barrier();                            // region R has been read
        rdx(SN{}, 0, x0);
        rdw(SN{}, w0);
        ffn_for<LA>([&](auto Q_) { dma(R_, p + NREG, Q_); });
        mma(1, x1, w1);
        weave(std::integral_constant<int, RX + RW>{}, std::integral_constant<int, LA>{});
    };
    // Pairs 0 .. NREG - 2 whole, and the first loads of the next.
    ffn_for<NREG - 1>([&](auto R_) { ffn_for<LPP>([&](auto Q_) { dma(R_, decltype(R_)::value, Q_); }); });
    ffn_for<LA>([&](auto Q_) { dma(std::integral_constant<int, NREG - 1>{}, NREG - 1, Q_); });
    __builtin_amdgcn_s_waitcnt(ffn_wait((NREG - 2) * LPP + LA));
    __builtin_amdgcn_s_barrier();
    rdx(std::integral_constant<int, 0>{}, 0, x0);
    rdw(std::integral_constant<int, 0>{}, w0);
    for (int p = 0; p < pairs; p += NREG) ffn_for<NREG>([&](auto R_) { pair(R_, p + decltype(R_)::value); });
    __builtin_amdgcn_s_waitcnt(ffn_wait(0));  // no load into LDS outlives its wave

    const Out out{a};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row = m0 + wm * TM + i * 16 + lr;
        if (row >= a.m) continue;
        if constexpr (G) {
#pragma unroll
            for (int j = 0; j < FN / 2; ++j)
                out.pair(row, n0 + wn * (TN / 2) + j * 16 + 4 * lq, acc[i][j], acc[i][j + FN / 2]);
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) out.one(row, n0 + wn * TN + j * 16 + 4 * lq, acc[i][j]);
        }
    }
}

// Place of tile t: groups of tile-rows, column by column inside a group.
template <int BM, int WO>
__device__ __forceinline__ void pipe_place(const FfnArgs& a, int64_t t, int64_t* m0, int64_t* n0) {
    const int64_t tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + WO - 1) / WO;
    const int64_t first = t / (PipeGroup * tiles_n) * PipeGroup;
    const int64_t size = tiles_m - first < PipeGroup ? tiles_m - first : PipeGroup;
    *m0 = (first + t % (PipeGroup * tiles_n) % size) * BM;
    *n0 = t % (PipeGroup * tiles_n) / size * WO;
}
// Tile of block `b` of `n`, a contiguous run on each XCD.
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t n) { return b % 8 * ((n + 7) / 8) + b / 8; }

template <class Out, class Z, bool XK = true, bool WK = true>
__global__ __launch_bounds__(Z::THREADS, Z::BLOCKS * Z::WAVES / 4) void ffn_pipe(FfnArgs a, int64_t tiles) {
    const int64_t t = xcd_run(blockIdx.x, tiles);
    if (t >= tiles) return;
    int64_t m0, n0;
    pipe_place<Z::BM, (Out::kGated ? Z::BN / 2 : Z::BN)>(a, t, &m0, &n0);
    pipe_tile<Out, Z, XK, WK>(a, m0, n0);
}

// `whole` tiles (a multiple of the CUs) in shape Z, the tiles after them as two of H
// each: a last round that would leave more than half of the CUs idle takes 0.6 of its
// time (4096 x 22016 over 4096 bf16, 1376 tiles: 661 -> 637 us).
template <class Out, class Z, class H>
__global__ __launch_bounds__(Z::THREADS, Z::BLOCKS * Z::WAVES / 4) void ffn_pipe_halves(FfnArgs a, int64_t whole,
                                                                                     int64_t halves) {
    static_assert(Z::THREADS == H::THREADS && Z::BM == H::BM && Z::BN == 2 * H::BN && Z::BLOCKS == H::BLOCKS, "halves");
    constexpr int WO = Out::kGated ? Z::BN / 2 : Z::BN;
    int64_t m0, n0;
    if ((int64_t)blockIdx.x < whole) {
        pipe_place<Z::BM, WO>(a, xcd_run(blockIdx.x, whole), &m0, &n0);
        pipe_tile<Out, Z, true, true>(a, m0, n0);
    } else {
        const int64_t t = xcd_run(blockIdx.x - whole, halves);
        if (t >= halves) return;
        pipe_place<Z::BM, WO>(a, whole + t / 2, &m0, &n0);
        n0 += t % 2 * (WO / 2);
        if (n0 < a.n) pipe_tile<Out, H, true, true>(a, m0, n0);
    }
}
#undef MM_LDS

// ---------------------------------------------------------------------------

// Rows that the pipelined forms take: 16-byte chunks that lie wholly inside a row,
// and a tile's rows within a resource's 31 bits.
inline bool ffn_chunked(const FfnArgs& a, int es) {
    const auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return al16(a.x) && al16(a.w) && a.ldx % 16 == 0 && a.ldw % 16 == 0 && a.k * es % 16 == 0 &&
           a.ldx < (1 << 22) && a.ldw < (1 << 22);
}

// 8 stages in LDS from 32 on, unless the last turn of the ring would be more than a
// twelfth in vain or, of 32 tokens (12 KB a stage), CUs have more than a tile; 4 otherwise.
// us, 4 and 8: f16 1 by 8192 rows, 16 stages 7.7 and 7.7, 24 10.0 and 9.8, 28 11.0 and
// 11.2, 32 12.0 and 12.0, 40 14.3 and 14.1, 64 30.2 and 28.9, 86 38.8 and 36.0; 1 by 1200,
// 24 5.1 and 5.2, 28 5.3 and 5.6, 32 6.7 and 5.7, 63 10.7 and 7.8; f32 16 by 4096, 24 7.5 and
// 7.1, 32 8.7 and 8.3, 128 38.0 and 30.7; 1 by 22016, 32 35.4 and 36.4, 64 67.8 and 65.6;
// codes 1 by 22016, 16 15.0 and 17.8, 32 35.0 and 34.0; 13 by 4099, 43 in turns of 48 11.4
// and 13.2, but 32 8.0 and 9.9; f32 32 by 4096, 128 44.9 and 38.1, by 22016, 64 91.5 and
// 104.9.
template <class Out, int FM>
hipError_t run_ffn_thin(const FfnArgs& a, hipStream_t s) {
    constexpr int XR = ThinShape<FM>::XR, WO = Out::kGated ? TRows / 2 : TRows, es = sizeof(typename Out::E::store_t);
    int tiles_m = (int)((a.m + XR - 1) / XR);
    const int64_t tiles = (int64_t)tiles_m * ((a.n + WO - 1) / WO);
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles_m};
    const int64_t stages = (a.k * es + TStage - 1) / TStage;
    const void* fn = reinterpret_cast<const void*>(&ffn_thin<Out, FM, 4>);
    if (stages >= 32 && ((stages + 7) / 8 * 8 - stages) * 12 <= stages && (FM == 1 || tiles <= 256))
        fn = reinterpret_cast<const void*>(&ffn_thin<Out, FM, 8>);
    return hipLaunchKernel(fn, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(64 * TWaves), args, 0, s);
}

template <class Out, class Z>
int64_t pipe_tiles(const FfnArgs& a) {
    constexpr int WO = Out::kGated ? Z::BN / 2 : Z::BN;
    return (a.m + Z::BM - 1) / Z::BM * ((a.n + WO - 1) / WO);
}
template <class Out, class Z, bool XK = true, bool WK = true>
hipError_t run_ffn_pipe(const FfnArgs& a, hipStream_t s) {
    int64_t tiles = pipe_tiles<Out, Z>(a);
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_pipe<Out, Z, XK, WK>),
                           dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(Z::THREADS), args, XK && WK ? Z::LDS : 0, s);
}
// Shape Z, with the tiles of a last round that fills no more than half of the CUs as
// halves H.
template <class Out, class Z, class H>
hipError_t run_ffn_pipe_halves(const FfnArgs& a, hipStream_t s) {
    const int64_t tiles = pipe_tiles<Out, Z>(a);
    int64_t whole = tiles / 256 * 256, halves = 2 * (tiles - whole);
    if (halves == 0 || halves > 256) return run_ffn_pipe<Out, Z>(a, s);
    void* args[] = {const_cast<FfnArgs*>(&a), &whole, &halves};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_pipe_halves<Out, Z, H>),
                           dim3((unsigned)(whole + (halves + 7) / 8 * 8)), dim3(Z::THREADS), args,
                           Z::LDS > H::LDS ? Z::LDS : H::LDS, s);
}

// The pipelined forms: tokens and rows of W of a tile, tiles at a time on the 256
// CUs, and what a round of them costs in us, for each 128 bytes of k and at its
// start. From 150 products of 1 to 8192 tokens in bf16 and codes, each in every form;
// the form with the lowest sum of rounds is within 3% of the fastest one in the
// mean. Both sides of some borders (us, all from one run): 48 tokens by 22016 x 4096
// bf16, 64 x 128 tiles 43.9, 64 x 64 47.5, 128 x 128 45.1; 512 by 2816 x 2048 codes, 64 x
// 128 9.4, 64 x 64 10.6, 128 x 128 13.0; 1024 by 22016 x 4096 bf16, 256 x 256 with its last
// round in halves 173, 256 x 128 182; 2048 by the same, 329 and 354; 32 by 1152 x 1792
// bf16, 32 x 16 5.4, 64 x 64 7.5. Up to 16 tokens take the thinnest: 1 by 22016 x 4096
// f16 35.0, 64 x 128 38.6; 1 by 8192 x 11008, 35.1, 64 x 64 51.1; 16 by 28672 x 4096 codes,
// 25.6, 64 x 64 26.0.
struct FfnForm {
    int tokens, rows, at_a_time;
    float pair_us, round_us;
};
constexpr FfnForm kFfnForms[] = {
    {16, 16, 0, 0.f, 0.f},         {32, 16, 512, 0.257f, 0.60f},   {64, 64, 256, 0.300f, 1.93f},
    {64, 128, 256, 0.320f, 2.26f}, {128, 128, 256, 0.607f, 2.15f}, {256, 128, 256, 0.956f, 3.35f},
    {256, 256, 256, 1.593f, 7.15f},
};
constexpr int kForms = sizeof kFfnForms / sizeof *kFfnForms;
inline int ffn_form(int64_t m, int64_t rows, int64_t bytes) {
    if (m <= 16) return 0;
    const float pairs = (float)((bytes + 127) / 128);
    int best = -1;
    float least = 0.f;
    for (int i = 1; i < kForms; ++i) {
        const FfnForm& f = kFfnForms[i];
        const int64_t tiles = ((m + f.tokens - 1) / f.tokens) * ((rows + f.rows - 1) / f.rows);
        const int64_t last = tiles % f.at_a_time;
        float us = (float)((tiles + f.at_a_time - 1) / f.at_a_time) * (pairs * f.pair_us + f.round_us);
        if (i == kForms - 1 && last > 0 && last <= f.at_a_time / 2)  // halves
            us -= pairs * (f.pair_us - kFfnForms[i - 1].pair_us) + f.round_us - kFfnForms[i - 1].round_us;
        if ((best < 0 || us < least) && tiles < (1 << 22)) {  // (a grid holds fewer than 2^32 threads)
            best = i;
            least = us;
        }
    }
    return best < 0 ? kForms - 1 : best;
}

// A product in the form that suits its size; the receipt's variant names it.
template <class Out>
hipError_t run_ffn(const FfnArgs& a, hipStream_t s, Launched* L) {
    using E = typename Out::E;
    constexpr int es = sizeof(typename E::store_t);
    static_assert(E::code != 0, "f32 has a choice of its own");
    if constexpr (E::code != 3) {  // codes always are
        if (!ffn_chunked(a, es)) return run_ffn_tile<Out>(a, s);
    }
    const int64_t rows = Out::kGated ? 2 * a.n : a.n;
    const int form = ffn_form(a.m, rows, a.k * es);
    L->variant = kFfnForms[form].tokens + 4096 * kFfnForms[form].rows;
    switch (form) {
        case 0: return run_ffn_thin<Out, 1>(a, s);
        case 1: return run_ffn_thin<Out, 2>(a, s);
        case 2: return run_ffn_pipe<Out, PipeShape<2, 2, 2, 2, 4>>(a, s);
        case 3: return run_ffn_pipe<Out, PipeShape<2, 4, 2, 2, 4>>(a, s);
        case 4: return run_ffn_pipe<Out, PipeShape<2, 4, 4, 2, 4>>(a, s);
        case 5: return run_ffn_pipe<Out, PipeShape<4, 2, 4, 4, 3>>(a, s);
        default: return run_ffn_pipe_halves<Out, PipeShape<2, 4, 8, 4, 2>, PipeShape<4, 2, 4, 4, 3>>(a, s);
    }
}

}  // namespace mmk
