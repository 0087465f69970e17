// Gated products of f32 rows in three bf16 parts (ffn_tile.hpp): forms whose waves part
// the fragments themselves, and the choice among all of f32's forms.
#pragma once

#include "ffn_pipe.hpp"

namespace mmk {

// The five small products, smallest first: parts of w and of x.
constexpr int kPartW[5] = {2, 0, 1, 1, 0}, kPartX[5] = {0, 2, 1, 0, 1};

__device__ __forceinline__ void part8(const float (&e)[8], u32x4 (&out)[3], uint32_t& lost) {
    uint32_t w[3][4];
    parts_of<TF32, 8>(e, w, lost);
#pragma unroll
    for (int q = 0; q < 3; ++q) out[q] = u32x4{w[q][0], w[q][1], w[q][2], w[q][3]};
}

__device__ __forceinline__ void part8(const u32x4 (&r)[2], u32x4 (&out)[3], uint32_t& lost) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __uint_as_float(r[i / 4][i % 4]);
    part8(e, out, lost);
}

// One step of 32 of k: the six products of FM x FN fragments. `x(i, f)` and `w(j, f)`
// give a fragment's parts.
template <int FM, int FN>
struct PartsAcc {
    f32x4 acc[FM][FN], low[FM][FN];  // upper parts; the small products
    uint32_t lost = 0;               // (parts_of)
    __device__ __forceinline__ PartsAcc() {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = low[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    template <class X, class W>
    __device__ __forceinline__ void step(X x, W w) {
        u32x4 fx[FM][3], fw[3];
#pragma unroll
        for (int i = 0; i < FM; ++i) x(i, fx[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            w(j, fw);
#pragma unroll
            for (int q = 0; q < 5; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i) low[i][j] = step_mma<TBF16>(fw[kPartW[q]], fx[i][kPartX[q]], low[i][j]);
#pragma unroll
            for (int i = 0; i < FM; ++i) acc[i][j] = step_mma<TBF16>(fw[0], fx[i][0], acc[i][j]);
        }
    }
};

// ---------------------------------------------------------------------------
// Rows of whole 16-byte chunks through the regions of ffn_pipe, two of them (a pair's
// 128 bytes are one step): LDS holds the raw 4 bytes an element, loads go there without
// a register, and each wave parts the fragments that it reads. Blocks share a CU: one's
// loads and barriers fall into the others' arithmetic. Bound by vector issue: parting is
// 192 of the 227 vector instructions a wave issues for 24 matrix instructions.
// ---------------------------------------------------------------------------
#define MM_LDS(p) ((__attribute__((address_space(3))) void*)(p))
template <class Out, class Z>
__global__ __launch_bounds__(Z::THREADS, 3) void ffn_pipe_f32(FfnArgs a, int64_t tiles) {
    static_assert(Out::kGated && Z::WAVES == 4 && 3 * Z::LDS <= 160 * 1024, "three blocks of a CU");
    constexpr int BM = Z::BM, FM = Z::FM, FN = Z::FN, NREG = Z::NREG, TM = 16 * FM, TN = 16 * FN, WO = Z::BN / 2;
    const int64_t t = xcd_run(blockIdx.x, tiles);
    if (t >= tiles) return;
    int64_t m0, n0;
    pipe_place<BM, WO>(a, t, &m0, &n0);
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / Z::WN, wn = w % Z::WN, lr = lane & 15, lq = lane >> 4;
    const int64_t bytes = a.k * 4;
    const int chunks = (int)(bytes / 16), pairs = (chunks + 7) / 8;
    const int ldx = (int)a.ldx, ldw = (int)a.ldw;
    const int64_t xrows = a.m - m0 < BM ? a.m - m0 : BM, wrows = a.n - n0 < WO ? a.n - n0 : WO;
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, m0, a.ldx, xrows, bytes);
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w, n0, a.ldw, wrows, bytes);
    const __amdgpu_buffer_rsrc_t ru = rows_rsrc(a.w, n0 + a.n, a.ldw, wrows, bytes);
    // A load covers 8 rows, the lane the chunk that belongs at slot lane % 8.
    const int dch = (lane & 7) ^ (lane >> 3);
    const int vox = (lane >> 3) * ldx + dch * 16, vow = (lane >> 3) * ldw + dch * 16;
    auto issue = [&](auto R_, int p) {
        char* region = pipe_lds + decltype(R_)::value * Z::REGION;
        const bool live = p * 8 + dch < chunks;  // (chunks past k are zeros)
#pragma unroll
        for (int q = 0; q < Z::XI; ++q) {
            const int row = (w * Z::XI + q) * 8;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, MM_LDS(region + row * 128), 16, live ? (uint32_t)vox : kPastEnd,
                                                     row * ldx + p * 128, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < Z::WI; ++q) {
            const int row = (w * Z::WI + q) * 8;  // each wave column's rows are half gate, half up projection
            const int col = row / TN * (TN / 2) + row % (TN / 2);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(row % TN >= TN / 2 ? ru : rw, MM_LDS(region + (BM + row) * 128), 16,
                                                     live ? (uint32_t)vow : kPastEnd, col * ldw + p * 128, 0, 0);
        }
    };
    PartsAcc<FM, FN> s;
    const int f0 = lr * 128 + ((lq ^ (lr & 7)) << 4), f1 = lr * 128 + (((4 + lq) ^ (lr & 7)) << 4);  // (k in one order for both)
    ffn_for<NREG - 1>([&](auto R_) { issue(R_, decltype(R_)::value); });
    for (int p = 0; p < pairs; p += NREG) {  // (pairs past the last one are zeros)
        ffn_for<NREG>([&](auto R_) {
            constexpr int R = decltype(R_)::value;
            // Pair p + R has landed; the pair before it has been read by every wave.
            __builtin_amdgcn_s_waitcnt(ffn_wait((NREG - 2) * Z::LOADS));
            __builtin_amdgcn_s_barrier();
            issue(std::integral_constant<int, (R + NREG - 1) % NREG>{}, p + R + NREG - 1);
            const char* xs = pipe_lds + R * Z::REGION + wm * TM * 128;
            const char* ws = pipe_lds + R * Z::REGION + (BM + wn * TN) * 128;
            const auto read = [&](const char* rows, u32x4(&f)[3]) {
                const u32x4 r[2] = {*reinterpret_cast<const u32x4*>(rows + f0), *reinterpret_cast<const u32x4*>(rows + f1)};
                part8(r, f, s.lost);
            };
            s.step([&](int i, u32x4(&f)[3]) { read(xs + i * 2048, f); },
                   [&](int j, u32x4(&f)[3]) { read(ws + j * 2048, f); });
        });
    }
    __builtin_amdgcn_s_waitcnt(ffn_wait(0));  // no load into LDS outlives its wave
    const auto x_row = [&](int row, int i) {
        const int64_t r = m0 + wm * TM + i * 16 + row;
        return static_cast<const float*>(a.x) + (r < a.m ? r : a.m - 1) * (a.ldx / 4);
    };
    const auto w_row = [&](int row, int j) {
        const int64_t r = n0 + wn * (TN / 2) + j % (FN / 2) * 16 + row;
        return static_cast<const float*>(a.w) + ((r < a.n ? r : a.n - 1) + (j >= FN / 2 ? a.n : 0)) * (a.ldw / 4);
    };
    f32_join<1, true, true>(a.k, 0, parts_lost(s.lost), x_row, 1, w_row, 1, s.acc, s.low);
    const Out out{a};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row = m0 + wm * TM + i * 16 + lr;
        if (row >= a.m) continue;
#pragma unroll
        for (int j = 0; j < FN / 2; ++j)
            out.pair(row, n0 + wn * (TN / 2) + j * 16 + 4 * lq, s.acc[i][j], s.acc[i][j + FN / 2]);
    }
}
#undef MM_LDS

// ---------------------------------------------------------------------------
// Rows of any alignment, few tiles: each of a block's KS waves computes the whole tile
// of 16 FM x 16 FN over every KS-th step. Waves share nothing, so there is no LDS and no
// barrier on the way (bound by parting and multiplying in turn, about 150 TFLOP/s of f32
// with all CUs at work): fragments come straight into registers (8 elements of a row a
// lane, a row's 128 bytes by four lanes), the next step's as soon as a fragment has been
// parted. At the end the partial tiles meet in LDS, summed in the order of the waves.
// Loads go through buffer resources: pitches up to 2^24 bytes, of 64 rows.
// ---------------------------------------------------------------------------
template <class Out, int FM, int FN, int KS>
__global__ __launch_bounds__(64 * KS, 2) void ffn_waves_f32(FfnArgs a, int64_t tiles) {
    constexpr int BM = 16 * FM, WO = 8 * FN;
    static_assert(Out::kGated, "gated");
    const int64_t t = xcd_run(blockIdx.x, tiles);
    if (t >= tiles) return;
    int64_t m0, n0;
    pipe_place<BM, WO>(a, t, &m0, &n0);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Loads take a lane's row and chunk as an offset, a fragment and a step as a scalar one. Rows
    // past the end are zeros; a fragment that has none but those reads the first one's.
    const int ldx = (int)a.ldx, ldw = (int)a.ldw;
    const int64_t xrows = a.m - m0 < BM ? a.m - m0 : BM, wrows = a.n - n0 < WO ? a.n - n0 : WO;
    const __amdgpu_buffer_rsrc_t bx = rows_rsrc(a.x, m0, a.ldx, xrows, a.k * 4);
    const __amdgpu_buffer_rsrc_t bw = rows_rsrc(a.w, n0, a.ldw, wrows, a.k * 4);
    const __amdgpu_buffer_rsrc_t bu = rows_rsrc(a.w, n0 + a.n, a.ldw, wrows, a.k * 4);
    const int vox = lr * ldx + 32 * lq, vow = lr * ldw + 32 * lq;
    const auto at_x = [&](int i) { return i * 16 < xrows ? i * 16 * ldx : 0; };
    const auto at_w = [&](int j) { return j % (FN / 2) * 16 < wrows ? j % (FN / 2) * 16 * ldw : 0; };
    int at = kg * 128;  // bytes
    u32x4 rx[FM][2], rw[FN][2];
    const auto load = [](__amdgpu_buffer_rsrc_t rs, int vo, int so, u32x4(&r)[2]) {
        r[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, vo, so, 0));
        r[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, vo + 16, so, 0));
    };
    const auto load_x = [&](int i) { load(bx, vox, at_x(i) + at, rx[i]); };
    const auto load_w = [&](int j) { load(j < FN / 2 ? bw : bu, vow, at_w(j) + at, rw[j]); };
    PartsAcc<FM, FN> s;
    const auto step = [&](auto more_) {  // and the next one's loads, each as soon as its registers are free
        constexpr bool more = decltype(more_)::value;
        if constexpr (more) at += 128 * KS;
        s.step(
            [&](int i, u32x4(&f)[3]) {
                part8(rx[i], f, s.lost);
                if constexpr (more) load_x(i);
            },
            [&](int j, u32x4(&f)[3]) {
                part8(rw[j], f, s.lost);
                if constexpr (more) load_w(j);
            });
    };
    const int whole = (int)(a.k / 32);
    int left = whole > kg ? (whole - kg + KS - 1) / KS : 0;
    if (left > 0) {
#pragma unroll
        for (int i = 0; i < FM; ++i) load_x(i);
#pragma unroll
        for (int j = 0; j < FN; ++j) load_w(j);
        for (; left > 1; --left) step(std::true_type{});
        step(std::false_type{});
    }
    if (a.k % 32 && whole % KS == kg) {  // the step that k ends in: zeros behind it, in both operands
        const int valid = (int)(a.k - (int64_t)whole * 32) - 8 * lq;
        const auto part = [&](__amdgpu_buffer_rsrc_t rs, int vo, int so, u32x4(&r)[2]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                r[e / 4][e % 4] = __builtin_amdgcn_raw_buffer_load_b32(rs, e < valid ? vo + 4 * e : (int)kPastEnd, so, 0);
        };
#pragma unroll
        for (int i = 0; i < FM; ++i) part(bx, vox, at_x(i) + whole * 128, rx[i]);
#pragma unroll
        for (int j = 0; j < FN; ++j) part(j < FN / 2 ? bw : bu, vow, at_w(j) + whole * 128, rw[j]);
        step(std::false_type{});
    }
    const auto x_row = [&](int row, int i) {
        const int64_t r = m0 + i * 16 + row;
        return static_cast<const float*>(a.x) + (r < a.m ? r : a.m - 1) * (a.ldx / 4);
    };
    const auto w_row = [&](int row, int j) {
        const int64_t r = n0 + j % (FN / 2) * 16 + row;
        return static_cast<const float*>(a.w) + ((r < a.n ? r : a.n - 1) + (j >= FN / 2 ? a.n : 0)) * (a.ldw / 4);
    };
    f32_join<KS, true, true>(a.k, kg, parts_lost(s.lost), x_row, 1, w_row, 1, s.acc, s.low);
    __shared__ f32x4 sums[KS][FM * FN][64];
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) sums[kg][f][lane] = s.acc[f / FN][f % FN];
    __syncthreads();
    const Out out{a};
    for (int u = kg; u < FM * FN / 2; u += KS) {
        const int i = u / (FN / 2), j = u % (FN / 2), f = i * FN + j;
        f32x4 g = sums[0][f][lane], v = sums[0][f + FN / 2][lane];
#pragma unroll
        for (int q = 1; q < KS; ++q) {
            g += sums[q][f][lane];
            v += sums[q][f + FN / 2][lane];
        }
        if (m0 + i * 16 + lr < a.m) out.pair(m0 + i * 16 + lr, n0 + j * 16 + 4 * lq, g, v);
    }
}

template <class Out, class Z>
hipError_t run_pipe_f32(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->variant = Z::BM + 4096 * Z::BN;
    int64_t tiles = pipe_tiles<Out, Z>(a);
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_pipe_f32<Out, Z>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                           dim3(Z::THREADS), args, Z::LDS, s);
}
template <class Out, int FM, int FN, int KS>
hipError_t run_ffn_waves(const FfnArgs& a, hipStream_t s) {
    int64_t tiles = (a.m + 16 * FM - 1) / (16 * FM) * ((a.n + 8 * FN - 1) / (8 * FN));
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_waves_f32<Out, FM, FN, KS>),
                           dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(64 * KS), args, 0, s);
}

// The forms of f32 rows: tokens and rows of w of a tile, elements of k an iteration,
// tiles at a time on the 256 CUs; and what a round of them costs in us, for each
// iteration and at its start. From 150 products of 65 to 4096 tokens in every form; the
// one with the lowest sum of rounds is within 3% of the fastest in the mean (9% where
// rows are not whole 16-byte chunks); measured before parting looked for lost bits, which
// costs 64 x 64 by four waves up to a tenth and the others 1 to 7%. Few tokens take f32
// instructions, at 2/5 of the rate of the six products but with nothing to part. Both sides
// of some borders, us: 70 tokens by 1200 over 8000, thin 33.1, 32 x 32 57.6; 256 by the
// same, thin 73.7, 32 x 64 86.3, 32 x 32 112; 70 by 2816 over 2048, thin 21.0, 32 x 64 24.9;
// 70 by 24000 over 1000, 64 x 64 by four waves 48.1, through LDS 49.2, 64 x 128 51.9; 400
// by 22016 over 4096, 64 x 128 506, 64 x 64 through LDS 571, by four waves 587, 128 x 128
// 587; 509 by 2816 over 2048, 64 x 64 through LDS 58.9, by four waves 62.8, 128 x 128 126;
// 4096 by 8192 over 4096, 128 x 128 1438, 64 x 64 through LDS 1804. Taken although slower:
// by four waves, 64 x 64 through LDS beside it, 160 by 22016 over 4096 291 and 276, 160 by
// 8192 over 11008 323 and 310, 1000 by 1200 over 8000 229 and 216.
// Bound by arithmetic from 512 tokens on: 4096 x 8192 over 4096 runs at 191 TFLOP/s, six
// times that in the matrix units; 509 by 2816 over 2048 at 100, for 352 tiles of 512.
template <class Out>
hipError_t run_ffn_f32(const FfnArgs& a, hipStream_t s, Launched* L) {
    const bool chunked = ffn_chunked(a, 4);
    const auto us = [&](int tokens, int rows, int kt, int at_a_time, float step, float start) {
        const int64_t tiles = (a.m + tokens - 1) / tokens * ((2 * a.n + rows - 1) / rows);
        if (tokens < 128 && tiles >= (1 << 22)) return 3e38f;  // (a grid holds fewer than 2^32 threads)
        return (float)((tiles + at_a_time - 1) / at_a_time) * ((float)((a.k + kt - 1) / kt) * step + start);
    };
    const float big = us(128, 128, 32, 512, 2.6f, 14.f);
    const float mid = chunked ? us(64, 64, 32, 512, 0.9f, 1.f) : us(64, 64, 32, 512, 1.2f, 3.f);
    const bool near = a.ldx <= (1 << 24) && a.ldw <= (1 << 24);  // (a tile within a resource's 31 bits)
    const float four = near ? us(64, 64, 128, 256, 1.6f, 4.f) : 3e38f;
    // A tile alone on its CU runs at 5/8 of the speed of two.
    const bool pairs = (a.m + 63) / 64 * ((2 * a.n + 127) / 128) > 256;
    const float broad = chunked && pairs ? us(64, 128, 32, 256, 0.74f, 2.f) : 3e38f;
    const float eight = near ? us(32, 32, 256, 256, 1.78f, 0.8f) : 3e38f;
    const float wide = near ? us(32, 64, 256, 256, 2.55f, 2.f) : 3e38f;
    const float thin = chunked ? a.m <= 16 ? 0.f : us(32, TRows, 64, 256, 0.2f, 0.5f) : big;
    if (broad <= thin && broad <= big && broad <= mid && broad <= four && broad <= eight && broad <= wide)
        return run_pipe_f32<Out, PipeShape<2, 2, 2, 4, 2>>(a, s, L);
    if (chunked && thin <= big && thin <= mid && thin <= four && thin <= eight && thin <= wide) {
        L->variant = (a.m <= 16 ? 16 : 32) + 4096 * TRows;
        return a.m <= 16 ? run_ffn_thin<Out, 1>(a, s) : run_ffn_thin<Out, 2>(a, s);
    }
    if (eight <= big && eight <= mid && eight <= four && eight <= wide) return run_ffn_waves<Out, 2, 2, 8>(a, s);
    if (wide <= big && wide <= mid && wide <= four) return run_ffn_waves<Out, 2, 4, 8>(a, s);
    if (four <= big && four <= mid) return run_ffn_waves<Out, 4, 4, 4>(a, s);
    const TileArgs t{a.x, a.w, a.m, a.n, a.k, a.ldx / 4, a.ldw / 4, 0};
    if (big <= mid) return run_tile<Out, TileShape<TF32, 4, 4, 1, 1>, true, true>(t, a, s);
    if (!chunked) return run_tile<Out, TileShape<TF32, 2, 2, 1, 1>, true, true>(t, a, s);
    return run_pipe_f32<Out, PipeShape<2, 2, 2, 2, 2>>(a, s, L);
}

}  // namespace mmk
