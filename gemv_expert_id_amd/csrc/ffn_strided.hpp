// Products of the gradients in f32, C[i][j] = sum_p A(i, p) B(p, j): B stored by rows of p (as a
// weight is, for dpre . w), A by rows of i or, transposed, of p. Rows of any
// alignment.
//
// A lane fetches four neighbouring columns of eight rows of p in eight loads and takes
// them as its elements of four fragments: fragment j of B holds the columns 4 c + j, c =
// 0 .. 15. What a matrix instruction leaves in a lane are then four neighbouring columns,
// one of each fragment. So an operand stored the other way round needs neither LDS nor a
// transposition, only an order of the columns of its own. Columns that would pass the
// end repeat the last four (their sums are the same and are stored twice, or not at all).
// Each of a block's KS waves computes the whole tile over every KS-th step of 32 of p;
// the partial tiles meet in LDS at the end, summed in the order of the waves. Bound by
// parting and multiplying in turn: 2000 x 4098 over 10000 142 TFLOP/s, 145 transposed.
#pragma once

#include "ffn_f32.hpp"

namespace mmk {

struct RowFrag {  // 8 neighbouring elements of p of one row
    Pack<float, 8> v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const Pack<float, 8>*>(p); }
    __device__ __forceinline__ void load(const float* p, int valid) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.v[e] = e < valid ? p[e] : 0.f;
    }
    __device__ __forceinline__ void parts(u32x4 (&f)[3], uint32_t& lost) const { part8(v.v, f, lost); }
};
struct ColumnFrags {  // 4 neighbouring columns of 8 rows of p
    Pack<float, 4> v[8];
    __device__ __forceinline__ void load(const float* p, int64_t ld) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = *reinterpret_cast<const Pack<float, 4>*>(p + e * ld);
    }
    __device__ __forceinline__ void load(const float* p, int64_t ld, int valid) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (e < valid) v[e] = *reinterpret_cast<const Pack<float, 4>*>(p + e * ld);
            else v[e] = Pack<float, 4>{};
        }
    }
    __device__ __forceinline__ void parts(int j, u32x4 (&f)[3], uint32_t& lost) const {
        const float e[8] = {v[0].v[j], v[1].v[j], v[2].v[j], v[3].v[j], v[4].v[j], v[5].v[j], v[6].v[j], v[7].v[j]};
        part8(e, f, lost);
    }
};

// AT: A is stored by rows of p too (FM is 4). Tiles of 16 FM x 64.
template <bool AT, int FM, int KS>
__global__ __launch_bounds__(64 * KS, FM == 4 ? 1 : 2) void strided_f32(FfnArgs a, int64_t tiles) {
    constexpr int BM = 16 * FM;
    static_assert(!AT || FM == 4, "four columns of A a lane");
    const int64_t t = xcd_run(blockIdx.x, tiles);
    if (t >= tiles) return;
    int64_t m0, n0;
    pipe_place<BM, 64>(a, t, &m0, &n0);
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int kg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t ldx = a.ldx / 4, ldw = a.ldw / 4, p0 = kg * 32 + 8 * lq;
    const auto first = [](int64_t at, int64_t end) { return at + 4 <= end ? at : end - 4; };
    const auto w_col = [&](int c, int j) { return static_cast<const float*>(a.w) + first(n0 + 4 * c, a.n) + j; };
    const auto x_row = [&](int row, int i) {
        const int64_t r = m0 + i * 16 + row;
        return static_cast<const float*>(a.x) + (AT ? first(m0 + 4 * row, a.m) + i : (r < a.m ? r : a.m - 1) * ldx);
    };
    const float* w = w_col(lr, 0) + p0 * ldw;
    const float* x[AT ? 1 : FM];
#pragma unroll
    for (int i = 0; i < (AT ? 1 : FM); ++i) x[i] = x_row(lr, i) + p0 * (AT ? ldx : 1);
    f32x4 acc[FM][4], low[FM][4];  // upper parts; the small products
    uint32_t lost = 0;             // (parts_of)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = low[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    ColumnFrags rw;
    std::conditional_t<AT, ColumnFrags, RowFrag> rx[AT ? 1 : FM];
    const auto load_w = [&] {
        rw.load(w, ldw);
        w += 32 * KS * ldw;
    };
    const auto load_x = [&](int i) {
        if constexpr (AT) {
            rx[0].load(x[0], ldx);
            x[0] += 32 * KS * ldx;
        } else {
            rx[i].load(x[i]);
            x[i] += 32 * KS;
        }
    };
    const auto step = [&](auto more_) {  // and the next one's loads
        constexpr bool more = decltype(more_)::value;
        u32x4 fw[4][3], fx[3];
#pragma unroll
        for (int j = 0; j < 4; ++j) rw.parts(j, fw[j], lost);
        if constexpr (more) load_w();
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if constexpr (AT) rx[0].parts(i, fx, lost);
            else rx[i].parts(fx, lost);
            if constexpr (more) {
                if (!AT || i == FM - 1) load_x(i);
            }
#pragma unroll
            for (int q = 0; q < 5; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) low[i][j] = step_mma<TBF16>(fw[j][kPartW[q]], fx[kPartX[q]], low[i][j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = step_mma<TBF16>(fw[j][0], fx[0], acc[i][j]);
        }
    };
    const int whole = (int)(a.k / 32);
    int left = whole > kg ? (whole - kg + KS - 1) / KS : 0;
    if (left > 0) {
#pragma unroll
        for (int i = 0; i < (AT ? 1 : FM); ++i) load_x(i);
        load_w();
        for (; left > 1; --left) step(std::true_type{});
        step(std::false_type{});
    }
    if (a.k % 32 && whole % KS == kg) {  // the step that p ends in: zeros behind it, in both operands
        const int valid = (int)(a.k - (int64_t)whole * 32) - 8 * lq;
        if constexpr (AT) {
            rx[0].load(x[0], ldx, valid);
        } else {
#pragma unroll
            for (int i = 0; i < FM; ++i) rx[i].load(x[i], valid);
        }
        rw.load(w, ldw, valid);
        step(std::false_type{});
    }
    __shared__ f32x4 sums[KS][FM * 4][64];
    f32_join<KS, !AT, false>(a.k, kg, parts_lost(lost), x_row, ldx, w_col, ldw, acc, low);
#pragma unroll
    for (int f = 0; f < FM * 4; ++f) sums[kg][f][lane] = acc[f / 4][f % 4];
    __syncthreads();
    // Unit (i, e): row i of a lane's, element e of its four fragments.
    const PlainOut<TF32> out{a};
    for (int u = kg; u < FM * 4; u += KS) {
        const int i = u / 4, e = u % 4;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = reinterpret_cast<const float*>(&sums[0][i * 4 + j][lane])[e];
#pragma unroll
            for (int q = 1; q < KS; ++q) v[j] += reinterpret_cast<const float*>(&sums[q][i * 4 + j][lane])[e];
        }
        const int64_t c = n0 + 4 * (4 * lq + e), r = AT ? m0 + 4 * lr : m0 + i * 16 + lr;
        if (c < a.n && r < a.m) out.one(AT ? first(r, a.m) + i : r, first(c, a.n), f32x4{v[0], v[1], v[2], v[3]});
    }
}

template <bool AT, int FM, int KS>
hipError_t run_strided(const FfnArgs& a, hipStream_t s) {
    int64_t tiles = (a.m + 16 * FM - 1) / (16 * FM) * ((a.n + 63) / 64);
    void* args[] = {const_cast<FfnArgs*>(&a), &tiles};
    return hipLaunchKernel(reinterpret_cast<const void*>(&strided_f32<AT, FM, KS>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                           dim3(64 * KS), args, 0, s);
}

// The forms of f32 and what a round of their tiles costs in us, as for the rows of W
// (ffn_f32.hpp). Both sides of some borders, us: dpre . w 70 x 4098 over 10000, 32 x 64
// here 76.5, 16 x 64 122, 64 x 64 134, 32 x 32 through LDS 190; 2000 x 4098 by the same,
// 64 x 64 here 1156, 32 x 64 1235, 128 x 64 through LDS 1449; 2000 x 8000 over 1200, 128 x
// 64 287, 64 x 64 here 326; 600 x 500 over 8192, 32 x 64 58.9, 16 x 64 80.8, 64 x 64 109;
// 16 x 8000 over 1200, 16 x 64 8.3, 32 x 64 10.8, 32 x 32 11.8. dpre^T . x 2816 x 2048 over
// 2000, 64 x 64 here 169, 128 x 64 205; over 200, 42.7 and 29.3.
template <bool AT>
hipError_t run_f32_product(const FfnArgs& a, hipStream_t s) {
    const auto us = [&](int bm, int bn, int kt, int at_a_time, float step, float start) {
        const int64_t tiles = (a.m + bm - 1) / bm * ((a.n + bn - 1) / bn);
        if (bm < 128 && tiles >= (1 << 22)) return 3e38f;  // (a grid holds fewer than 2^32 threads)
        return (float)((tiles + at_a_time - 1) / at_a_time) * ((float)((a.k + kt - 1) / kt) * step + start);
    };
    const bool fours = a.n >= 4 && (!AT || a.m >= 4);
    const float big = us(128, 64, 32, 512, 1.7f, 5.f), mid = us(64, 64, 32, 512, 1.3f, 1.5f);
    const float four = !fours ? 3e38f : AT ? us(64, 64, 128, 256, 1.45f, 5.f) : us(64, 64, 128, 256, 1.7f, 2.f);
    const TileArgs t{a.x, a.w, a.m, a.n, a.k, a.ldx / 4, a.ldw / 4, 0};
    if constexpr (AT) {
        const bool few = (a.m + 31) / 32 * ((a.n + 31) / 32) <= 256;
        const float narrow = us(32, 32, 128, 256, 0.95f, 1.f);
        if (few && narrow <= big && narrow <= mid && narrow <= four)
            return run_tile<PlainOut<TF32>, TileShape<TF32, 1, 1, 1, 4>, false, false>(t, a, s);
    } else {
        const float one = !fours ? 3e38f : us(16, 64, 256, 256, 1.4f, 1.f);
        const float two = !fours ? 3e38f : us(32, 64, 256, 256, 1.75f, 1.5f);
        if (one <= big && one <= mid && one <= two && one <= four) return run_strided<false, 1, 8>(a, s);
        if (two <= big && two <= mid && two <= four) return run_strided<false, 2, 8>(a, s);
    }
    if (four <= big && four <= mid) return run_strided<AT, 4, 4>(a, s);
    if (big <= mid) return run_tile<PlainOut<TF32>, TileShape<TF32, 4, 2, 1, 1>, !AT, false>(t, a, s);
    return run_tile<PlainOut<TF32>, TileShape<TF32, 2, 2, 1, 1>, !AT, false>(t, a, s);
}

}  // namespace mmk
