// Tiled product of the feed-forward block, any length, pitch and alignment:
// sums of x [m, k] with the rows of W, W = [n, k] or, gated, [2n, k] with the
// gate's rows first.
//
// Block = 4 waves (2 x 2), tile 128 tokens x 128 rows of W, 64 bytes of k at a
// step, double-buffered in LDS: the next step's 16-byte chunks are fetched into
// registers before the current one is multiplied. Gated, a tile's 128 rows are
// 64 outputs: each wave's 64 rows are 32 of the gate and the same 32 of the up
// projection, so both sums of an output end in the same lane and the gate needs
// no exchange. LDS rows are 80 bytes apart: the 16 rows that a fragment read
// covers start in distinct banks.
#pragma once

#include "ffn.hpp"

namespace mmk {

constexpr int FT = 128;             // tile edge: tokens, rows of W
constexpr int FStep = 64;           // bytes of k at a step
constexpr int FPitch = FStep + 16;  // bytes between LDS rows
constexpr int FThreads = 256;

template <class S>
struct __attribute__((packed, aligned(sizeof(S)))) Unaligned16 {
    u32x4 v;
};

// 16 bytes of a row at byte `at`, zeros from byte `end` on.
template <class E>
__device__ __forceinline__ u32x4 row_chunk(const char* row, int64_t at, int64_t end) {
    using S = typename E::store_t;
    if (at + 16 <= end) return reinterpret_cast<const Unaligned16<S>*>(row + at)->v;
    u32x4 v = {0u, 0u, 0u, 0u};
    for (int i = 0; i < E::Elems16; ++i) {
        if (at + (i + 1) * (int)sizeof(S) > end) break;
        if constexpr (sizeof(S) == 4)
            v[i] = reinterpret_cast<const uint32_t*>(row + at)[i];
        else if constexpr (sizeof(S) == 2)
            v[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row + at)[i] << (16 * (i % 2));
        else
            v[i / 4] |= (uint32_t)reinterpret_cast<const uint8_t*>(row + at)[i] << (8 * (i % 4));
    }
    return v;
}

template <class Out>
__global__ __launch_bounds__(FThreads) void ffn_tile(FfnArgs a) {
    using E = typename Out::E;
    using Acc = typename AccOf<E>::type;
    constexpr bool G = Out::kGated;
    constexpr int FN = G ? FT / 2 : FT;  // outputs of a tile
    __shared__ __attribute__((aligned(16))) char xs[2][FT * FPitch];
    __shared__ __attribute__((aligned(16))) char ws[2][FT * FPitch];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, lr = lane & 15, lq = lane >> 4;
    const Out out{a};
    const int64_t tiles_n = (a.n + FN - 1) / FN, tiles = (a.m + FT - 1) / FT * tiles_n;
    const int64_t bytes = a.k * (int64_t)sizeof(typename E::store_t);
    const int64_t steps = (bytes + FStep - 1) / FStep;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m0 = t / tiles_n * FT, n0 = t % tiles_n * FN;
        // Chunks of this thread: rows tid / 4 and tid / 4 + 64, chunk tid % 4.
        const char* xr[2];
        const char* wr[2];
        int64_t xe[2], we[2];  // bytes of each row that exist
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = tid / 4 + 64 * u;
            const int64_t xrow = m0 + r;
            xe[u] = xrow < a.m ? bytes : 0;
            xr[u] = static_cast<const char*>(a.x) + (xrow < a.m ? xrow : 0) * a.ldx;
            int64_t col = n0 + r, wrow = col;
            if (G) {  // 32 rows of the gate, 32 of the up projection, twice
                col = n0 + (r >> 6) * 32 + (r & 31);
                wrow = col + ((r >> 5) & 1) * a.n;
            }
            we[u] = col < a.n ? bytes : 0;
            wr[u] = static_cast<const char*>(a.w) + (col < a.n ? wrow : 0) * a.ldw;
        }
        u32x4 xv[2], wv[2];
        auto fetch = [&](int64_t s) {
            const int64_t at = s * FStep + (tid & 3) * 16;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                xv[u] = row_chunk<E>(xr[u], at, xe[u]);
                wv[u] = row_chunk<E>(wr[u], at, we[u]);
            }
        };
        auto store = [&](int b) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = (tid / 4 + 64 * u) * FPitch + (tid & 3) * 16;
                *reinterpret_cast<u32x4*>(&xs[b][at]) = xv[u];
                *reinterpret_cast<u32x4*>(&ws[b][at]) = wv[u];
            }
        };
        Acc acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = Acc{0, 0, 0, 0};
        fetch(0);
        __syncthreads();  // the previous tile's readers are done
        store(0);
        __syncthreads();
        for (int64_t s = 0; s < steps; ++s) {
            const int cur = (int)(s & 1);
            const bool more = s + 1 < steps;
            if (more) fetch(s + 1);
            u32x4 xf[4], wf[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xf[i] = *reinterpret_cast<const u32x4*>(&xs[cur][(wm * 64 + i * 16 + lr) * FPitch + lq * 16]);
                wf[i] = *reinterpret_cast<const u32x4*>(&ws[cur][(wn * 64 + i * 16 + lr) * FPitch + lq * 16]);
            }
            // Lane: token lr of fragment i, rows 4 lq .. + 3 of W's fragment j.
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = step_mma<E>(wf[j], xf[i], acc[i][j]);
            if (more) store(cur ^ 1);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = m0 + wm * 64 + i * 16 + lr;
            if (row >= a.m) continue;
            if constexpr (G) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    out.pair(row, n0 + wn * 32 + j * 16 + 4 * lq, acc[i][j], acc[i][j + 2]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) out.one(row, n0 + wn * 64 + j * 16 + 4 * lq, acc[i][j]);
            }
        }
    }
}

inline int64_t ffn_tiles(const FfnArgs& a, bool gated) {
    const int64_t fn = gated ? FT / 2 : FT;
    return (a.m + FT - 1) / FT * ((a.n + fn - 1) / fn);
}

template <class Out>
hipError_t run_ffn_tile(const FfnArgs& a, hipStream_t s) {
    const int64_t tiles = ffn_tiles(a, Out::kGated);
    const unsigned grid = (unsigned)(tiles < (1 << 22) ? tiles : 1 << 22);
    void* args[] = {const_cast<FfnArgs*>(&a)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_tile<Out>), dim3(grid), dim3(FThreads), args, 0, s);
}

}  // namespace mmk
