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
// Few tokens: 16 FM tokens by 64 / KS rows of W, the contraction in stages of
// 256 bytes.
//
// W is read once, 256 contiguous bytes of a row at a time, and the tokens' pieces
// with it (from L2). A stage is four steps of matrix instructions. KS = 1: the four
// waves take 16 rows each and all four steps; KS = 2 and 4: 32 or 16 rows, the waves
// split the steps and are joined through LDS at the end, for the rows that would
// leave CUs idle otherwise. Chunk c of LDS row r lies at slot c ^ (r & 15), so the
// 16 rows of a fragment read cover all banks.
//
// Gated, a fragment's 16 rows are eight of the gate and the same eight of the up
// projection: the two sums of an output end 32 lanes apart.
// ---------------------------------------------------------------------------
constexpr int TStage = 256;  // bytes of k a stage
constexpr int TRing = 4;     // stages in LDS

template <int FM, int KS>
struct ThinShape {
    static constexpr int XR = 16 * FM;           // tokens
    static constexpr int WN = 4 / KS;            // waves along W's rows
    static constexpr int WR = 16 * WN;           // rows of W
    static constexpr int XI = FM, WI = WR / 16;  // loads of a wave and stage
    static constexpr int LOADS = XI + WI;
    static constexpr int BYTES = (XR + WR) * TStage;
    static constexpr int STEPS = 4 / KS;  // steps of a wave and stage
};

// Stage S of the ring: arrays of their own, so that the compiler sees that reads of
// one stage do not meet the loads in flight into others.
template <int BYTES, int S>
__device__ __forceinline__ char* thin_stage() {
    __shared__ __attribute__((aligned(1024))) char st[BYTES];
    return st;
}

template <class Out, int FM, int KS>
__global__ __launch_bounds__(256) void ffn_thin(FfnArgs a, int tiles_m) {
    using E = typename Out::E;
    using Acc = typename AccOf<E>::type;
    using Z = ThinShape<FM, KS>;
    constexpr bool G = Out::kGated;
    constexpr int WO = G ? Z::WR / 2 : Z::WR;  // outputs
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = w % Z::WN, ks = w / Z::WN, lr = lane & 15, lq = lane >> 4;
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
        for (int j = 0; j < Z::XI; ++j) {
            const int row = (w * Z::XI + j) * 4, c = c0 ^ (row & 12);
            const uint32_t at = st * 16 + c < chunks ? (uint32_t)(r4 * ldx + c * 16) : kPastEnd;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MM_LDS(base + row * TStage), 16, at,
                                                     row * ldx + st * TStage, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < Z::WI; ++j) {
            const int row = (w * Z::WI + j) * 4, c = c0 ^ (row & 12);
            const uint32_t at = st * 16 + c < chunks ? (uint32_t)(r4 * ldw + c * 16) : kPastEnd;
            const bool up = G && (row & 8);
            const int col = G ? (row >> 4) * 8 + (row & 7) : row;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ru : rw, MM_LDS(base + (Z::XR + row) * TStage), 16, at,
                                                     col * ldw + st * TStage, 0, 0);
        }
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
#pragma unroll
        for (int s = 0; s < Z::STEPS; ++s) {
            const int at = ((4 * (ks * Z::STEPS + s) + lq) ^ lr) * 16;
            const u32x4 wf = *reinterpret_cast<const u32x4*>(base + (Z::XR + wn * 16 + lr) * TStage + at);
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
        }
    };
    ffn_for<TRing - 1>([&](auto S_) { issue(S_, decltype(S_)::value); });
    for (int st = 0; st < stages; st += TRing) {
        ffn_for<TRing>([&](auto S_) {
            constexpr int s = decltype(S_)::value;
            // Stage st + s has landed; the stage before it has been read by every wave.
            __builtin_amdgcn_s_waitcnt(ffn_wait((TRing - 2) * Z::LOADS));
            __builtin_amdgcn_s_barrier();
            issue(std::integral_constant<int, (s + TRing - 1) % TRing>{}, st + s + TRing - 1);
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
    if constexpr (KS > 1) {
        __syncthreads();
        Acc* part = reinterpret_cast<Acc*>(thin_stage<Z::BYTES, 0>());
        static_assert((KS - 1) * Z::WN * FM * 64 * 16 <= Z::BYTES, "partial sums fit a stage");
        if (ks > 0) {
#pragma unroll
            for (int i = 0; i < FM; ++i) part[(((ks - 1) * Z::WN + wn) * FM + i) * 64 + lane] = acc[i];
        }
        __syncthreads();
        if (ks > 0) return;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int q = 1; q < KS; ++q) acc[i] += part[(((q - 1) * Z::WN + wn) * FM + i) * 64 + lane];
    }
    const Out out{a};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row = m0 + i * 16 + lr;
        if constexpr (G) {
            Acc u;
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] = __shfl_xor(acc[i][q], 32, kWave);
            if (lq < 2 && row < a.m) out.pair(row, n0 + wn * 8 + 4 * lq, acc[i], u);
        } else {
            if (row < a.m) out.one(row, n0 + wn * 16 + 4 * lq, acc[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Many tokens: 32 TF tokens by 32 TF rows of W, 4 waves of 16 TF x 16 TF each, the
// contraction in pairs of 64-byte steps, as in the paired-stage GEMM.
//
// A region of LDS holds 128 bytes of every row of a tile (chunk c of row r at slot
// c ^ (r & 7)); a load covers 8 rows. Of a pair's two steps, the second's barrier
// frees its region for the pair NREG later, whose loads go out between the matrix
// instructions of the next two half steps. Gated, a wave's 16 TF rows of W are half
// gate, half up projection, so an output's two sums end in one lane.
// ---------------------------------------------------------------------------
template <int TF, int NREG>
struct PipeShape {
    static constexpr int BM = 32 * TF;             // tile edge
    static constexpr int WT = 16 * TF;             // wave tile edge
    static constexpr int OP = BM * 128;            // bytes of an operand and region
    static constexpr int REGION = 2 * OP;
    static constexpr int LOADS = BM / 32;          // loads of a wave, operand and pair
    static constexpr size_t LDS = (size_t)NREG * REGION;
};

constexpr int PipeGroup = 4;  // tile-rows of a group: neighbours in time share W through L2

template <class Out, int TF, int NREG>
__global__ __launch_bounds__(256, TF == 8 || NREG > 2 ? 1 : 2) void ffn_pipe(FfnArgs a) {
    using E = typename Out::E;
    using Acc = typename AccOf<E>::type;
    using Z = PipeShape<TF, NREG>;
    constexpr bool G = Out::kGated;
    constexpr int BM = Z::BM, WT = Z::WT, HF = TF / 2, LD = Z::LOADS, LPP = 2 * LD;
    constexpr int WO = G ? BM / 2 : BM;                      // outputs of a tile
    constexpr int MPR = HF * TF / LD;                        // matrix instructions between loads
    extern __shared__ __attribute__((aligned(1024))) char pipe_lds[];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w >> 1, wn = w & 1, lr = lane & 15, lq = lane >> 4;

    // Groups of tile-rows, column by column inside a group, a contiguous run on each XCD.
    const int64_t tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + WO - 1) / WO, tiles = tiles_m * tiles_n;
    const int64_t per_xcd = (tiles + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    if (t >= tiles) return;
    const int64_t first = t / (PipeGroup * tiles_n) * PipeGroup;
    const int64_t size = tiles_m - first < PipeGroup ? tiles_m - first : PipeGroup;
    const int64_t m0 = (first + t % (PipeGroup * tiles_n) % size) * BM;
    const int64_t n0 = t % (PipeGroup * tiles_n) / size * WO;

    const int64_t bytes = a.k * (int64_t)sizeof(typename E::store_t);
    const int chunks = (int)(bytes / 16);
    const int pairs = ((chunks + 7) / 8 + NREG - 1) / NREG * NREG;
    const int ldx = (int)a.ldx, ldw = (int)a.ldw;
    // This wave loads rows w BM / 4 .. of both operands; gated, waves 0 and 2 the
    // gate's rows of wave columns 0 and 1, waves 1 and 3 the up projection's.
    constexpr int WL = BM / 4;
    const int64_t xat = m0 + w * WL, wat = G ? n0 + (w >> 1) * WL : n0 + w * WL;
    const int64_t xrows = a.m - xat < WL ? a.m - xat : WL, wrows = a.n - wat < WL ? a.n - wat : WL;
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, xrows > 0 ? xat : 0, a.ldx, xrows, bytes);
    const __amdgpu_buffer_rsrc_t rw =
        rows_rsrc(a.w, wrows > 0 ? wat + (G && (w & 1) ? a.n : 0) : 0, a.ldw, wrows, bytes);
    const int dch = (lane & 7) ^ (lane >> 3);
    const int vox = (lane >> 3) * ldx + dch * 16, vow = (lane >> 3) * ldw + dch * 16;

    // Load q (operand q % 2, its load q / 2) of pair p into region R.
    auto dma = [&](auto R_, int p, auto Q_) {
        constexpr int R = decltype(R_)::value, q = decltype(Q_)::value, j = q / 2;
        const bool live = p * 8 + dch < chunks;
        char* at = pipe_lds + R * Z::REGION + (q % 2) * Z::OP + (w * WL + j * 8) * 128;
        if constexpr (q % 2 == 0)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MM_LDS(at), 16, live ? (uint32_t)vox : kPastEnd,
                                                     j * 8 * ldx + p * 128, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, MM_LDS(at), 16, live ? (uint32_t)vow : kPastEnd,
                                                     j * 8 * ldw + p * 128, 0, 0);
    };
    Acc acc[TF][TF];
#pragma unroll
    for (int i = 0; i < TF; ++i)
#pragma unroll
        for (int j = 0; j < TF; ++j) acc[i][j] = Acc{0, 0, 0, 0};
    const int f0 = lr * 128 + ((lq ^ (lr & 7)) << 4), f1 = lr * 128 + (((4 + lq) ^ (lr & 7)) << 4);
    // Step S (region S / 2, half S % 2): x fragments of half hh of the wave's rows, all of W's.
    auto rdx = [&](auto S_, int hh, u32x4 (&f)[HF]) {
        constexpr int s = decltype(S_)::value;
        const char* p = pipe_lds + (s / 2) * Z::REGION + (wm * WT + hh * (WT / 2)) * 128 + (s % 2 ? f1 : f0);
#pragma unroll
        for (int i = 0; i < HF; ++i) f[i] = *reinterpret_cast<const u32x4*>(p + i * 16 * 128);
    };
    auto rdw = [&](auto S_, u32x4 (&f)[TF]) {
        constexpr int s = decltype(S_)::value;
        const char* p = pipe_lds + (s / 2) * Z::REGION + Z::OP + wn * WT * 128 + (s % 2 ? f1 : f0);
#pragma unroll
        for (int j = 0; j < TF; ++j) f[j] = *reinterpret_cast<const u32x4*>(p + j * 16 * 128);
    };
    auto mma = [&](int hh, const u32x4 (&fx)[HF], const u32x4 (&fw)[TF]) {
#pragma unroll
        for (int i = 0; i < HF; ++i)
#pragma unroll
            for (int j = 0; j < TF; ++j) acc[hh * HF + i][j] = step_mma<E>(fw[j], fx[i], acc[hh * HF + i][j]);
    };
    // Fragment reads first, then a load after every MPR matrix instructions.
    auto weave = [&](auto READS) {
        __builtin_amdgcn_sched_group_barrier(0x100, decltype(READS)::value, 0);
#pragma unroll
        for (int q = 0; q < LD; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, MPR, 0);
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    u32x4 x0[HF], x1[HF], w0[TF], w1[TF];
    // Both steps of pair p, in region R. The first half of step 0 sends out the
    // second half of pair p + NREG - 1, the second half of step 1 the first half of
    // pair p + NREG.
    auto pair = [&](auto R_, int p) {
        constexpr int R = decltype(R_)::value, RP = (R + NREG - 1) % NREG, RN = (R + 1) % NREG;
        using S0 = std::integral_constant<int, 2 * R>;
        using S1 = std::integral_constant<int, 2 * R + 1>;
        using SN = std::integral_constant<int, 2 * RN>;
        rdx(S0{}, 1, x1);
        ffn_for<LD>([&](auto Q_) {
            dma(std::integral_constant<int, RP>{}, p + NREG - 1, std::integral_constant<int, LD + decltype(Q_)::value>{});
        });
        mma(0, x0, w0);
        weave(std::integral_constant<int, HF>{});
        rdx(S1{}, 0, x0);
        rdw(S1{}, w1);
        mma(1, x1, w0);
        __builtin_amdgcn_sched_group_barrier(0x100, HF + TF, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, HF * TF, 0);
        __builtin_amdgcn_sched_barrier(0);
        rdx(S1{}, 1, x1);
        mma(0, x0, w1);
        __builtin_amdgcn_sched_group_barrier(0x100, HF, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, HF * TF, 0);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(ffn_wait((NREG - 2) * LPP));  // pair p + 1 has landed
        __builtin_amdgcn_s_barrier();                            // region R has been read
        rdx(SN{}, 0, x0);
        rdw(SN{}, w0);
        ffn_for<LD>([&](auto Q_) { dma(R_, p + NREG, Q_); });
        mma(1, x1, w1);
        weave(std::integral_constant<int, HF + TF>{});
    };
    // Pairs 0 .. NREG - 2 whole, and the first half of the next.
    ffn_for<NREG - 1>([&](auto R_) { ffn_for<LPP>([&](auto Q_) { dma(R_, decltype(R_)::value, Q_); }); });
    ffn_for<LD>([&](auto Q_) { dma(std::integral_constant<int, NREG - 1>{}, NREG - 1, Q_); });
    __builtin_amdgcn_s_waitcnt(ffn_wait((NREG - 2) * LPP + LD));
    __builtin_amdgcn_s_barrier();
    rdx(std::integral_constant<int, 0>{}, 0, x0);
    rdw(std::integral_constant<int, 0>{}, w0);
    for (int p = 0; p < pairs; p += NREG) ffn_for<NREG>([&](auto R_) { pair(R_, p + decltype(R_)::value); });
    __builtin_amdgcn_s_waitcnt(ffn_wait(0));  // no load into LDS outlives its wave

    const Out out{a};
#pragma unroll
    for (int i = 0; i < TF; ++i) {
        const int64_t row = m0 + wm * WT + i * 16 + lr;
        if (row >= a.m) continue;
        if constexpr (G) {
#pragma unroll
            for (int j = 0; j < HF; ++j)
                out.pair(row, n0 + wn * (WT / 2) + j * 16 + 4 * lq, acc[i][j], acc[i][j + HF]);
        } else {
#pragma unroll
            for (int j = 0; j < TF; ++j) out.one(row, n0 + wn * WT + j * 16 + 4 * lq, acc[i][j]);
        }
    }
}
#undef MM_LDS

// ---------------------------------------------------------------------------

// Rows that the pipelined forms take: 16-byte chunks that lie wholly inside a row,
// and a tile's rows within a resource's 31 bits.
inline bool ffn_chunked(const FfnArgs& a, int es) {
    const auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return al16(a.x) && al16(a.w) && a.ldx % 16 == 0 && a.ldw % 16 == 0 && a.k * es % 16 == 0 &&
           a.ldx < (1 << 24) && a.ldw < (1 << 24);
}

template <class Out, int FM, int KS>
hipError_t run_ffn_thin(const FfnArgs& a, hipStream_t s) {
    using Z = ThinShape<FM, KS>;
    constexpr int WO = Out::kGated ? Z::WR / 2 : Z::WR;
    int tiles_m = (int)((a.m + Z::XR - 1) / Z::XR);
    const int64_t tiles = (int64_t)tiles_m * ((a.n + WO - 1) / WO);
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles_m};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_thin<Out, FM, KS>),
                           dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(256), args, 0, s);
}

template <class Out, int TF, int NREG>
hipError_t run_ffn_pipe(const FfnArgs& a, hipStream_t s) {
    using Z = PipeShape<TF, NREG>;
    constexpr int WO = Out::kGated ? Z::BM / 2 : Z::BM;
    const int64_t tiles = (a.m + Z::BM - 1) / Z::BM * ((a.n + WO - 1) / WO);
    void* args[] = {const_cast<FfnArgs*>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_pipe<Out, TF, NREG>),
                           dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(256), args, Z::LDS, s);
}

template <class Out>
hipError_t run_ffn_thin(const FfnArgs& a, int fm, int ks, hipStream_t s) {
#define MM_THIN(F, K) \
    if (fm == F && ks == K) return run_ffn_thin<Out, F, K>(a, s);
    MM_THIN(1, 1) MM_THIN(2, 1) MM_THIN(3, 1) MM_THIN(4, 1)
    MM_THIN(1, 2) MM_THIN(2, 2) MM_THIN(3, 2) MM_THIN(4, 2)
    MM_THIN(1, 4) MM_THIN(2, 4) MM_THIN(3, 4) MM_THIN(4, 4)
#undef MM_THIN
    return hipErrorInvalidValue;
}

// The form for a product, reported as the receipt's variant.
template <class Out>
hipError_t run_ffn(const FfnArgs& a, hipStream_t s, Launched* L) {
    using E = typename Out::E;
    if constexpr (E::code != 3) {  // codes always are
        if (!ffn_chunked(a, sizeof(typename E::store_t)) || (E::code == 0 && a.m > 64)) return run_ffn_tile<Out>(a, s);
    }
    const int64_t rows = Out::kGated ? 2 * a.n : a.n;
    if (a.m <= 64) {
        const int fm = (int)((a.m + 15) / 16);
        const int ks = rows > 64 * 255 ? 1 : rows > 32 * 255 ? 2 : 4;
        L->variant = fm + 256 * ks;
        return run_ffn_thin<Out>(a, fm, ks, s);
    }
    if constexpr (E::code != 0) {
        const int64_t big = ((a.m + 255) / 256) * ((rows + 255) / 256);
        if (big >= 192) {
            L->variant = 256 + 2;
            return run_ffn_pipe<Out, 8, 2>(a, s);
        }
        const int64_t mid = ((a.m + 127) / 128) * ((rows + 127) / 128);
        if (mid > 256) {
            L->variant = 128 + 2;
            return run_ffn_pipe<Out, 4, 2>(a, s);
        }
        L->variant = 128 + 4;
        return run_ffn_pipe<Out, 4, 4>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mmk
