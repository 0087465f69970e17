// Tiled products of the feed-forward block for f32, and for 16-bit rows of any
// alignment: C[i][j] = sum_p A(i, p) B(j, p), each operand with p contiguous
// (element (i, p) at i * ld + p) or strided (at p * ld + i).
//
// f32 operands enter the matrix instructions as three bf16 parts (8 + 8 + 8 bits,
// exact down to 2^-133) and six products of parts, 00 01 10 11 02 20; what is left
// out is below 2^-24 of a product. 16x16x32 bf16 takes 16 cycles, f32 instructions
// 256 for the same tile: 96 for the six. The products of upper parts have an
// accumulator of their own, so the small ones are not rounded away. 16-bit operands
// are one part.
//
// Block = 4 waves (2 x 2), tile 32 F x 32 F, 32 elements of k at a step, staged
// through registers: the next step is fetched before the current one is multiplied.
// A contiguous operand is fetched in 16-byte pieces at any address, a strided one in
// blocks of F k-rows by 4 columns, which registers transpose on the way to LDS.
// Rows and columns past the end repeat the last one (their sums are not stored);
// elements of k past the end are zeros in both operands. LDS rows are 80 bytes
// apart: the 16 rows that a fragment read covers start in distinct banks.
#pragma once

#include "ffn.hpp"

namespace mmk {

constexpr int AStep = 32;     // elements of k at a step
constexpr int APitch = 80;    // bytes between LDS rows (64 of them used)
constexpr int AThreads = 256;

template <class S, int N>
struct __attribute__((packed, aligned(sizeof(S)))) Pack {
    S v[N];
};

struct TileArgs {
    const void* a;
    const void* b;
    int64_t m, n, k;   // C is m x n; gated, n outputs from 2n rows of B
    int64_t lda, ldb;  // elements
    int32_t tiles_n;
};

// Parts of a type's elements in the matrix instructions.
template <class T> constexpr int kParts = T::code == 0 ? 3 : 1;
template <class T> using MmaOf = std::conditional_t<T::code == 1, TF16, TBF16>;

// N elements as their parts, two to a register.
template <class T, int N>
__device__ __forceinline__ void parts_of(const typename T::store_t (&e)[N], uint32_t (&out)[kParts<T>][N / 2]) {
    if constexpr (T::code == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float lo = e[2 * i], hi = e[2 * i + 1];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                out[q][i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
                lo -= __uint_as_float(__float_as_uint(lo) & 0xFFFF0000u);
                hi -= __uint_as_float(__float_as_uint(hi) & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[0][i] = (uint32_t)e[2 * i] | ((uint32_t)e[2 * i + 1] << 16);
    }
}

// One operand's share of a thread: R = 32 F rows by 32 elements of k.
template <class T, int F, bool KC>
struct TileOperand {
    using S = typename T::store_t;
    static constexpr int R = 32 * F;
    static constexpr int V = KC ? T::Elems16 : 4;              // elements of a load
    static constexpr int N = KC ? R * AStep / V / AThreads : F;  // loads
    static constexpr int PLANE = R * APitch;                   // bytes of one part in LDS
    Pack<S, V> v[N];
    const S* p[KC ? N : 4];  // row starts; or the four columns (p[0] alone while they are neighbours)
    int64_t ld;
    bool split;  // strided: the columns are fetched one by one

    // `row(r)`: the operand's row that tile row r stands for, already inside it.
    template <class Row>
    __device__ __forceinline__ void init(const void* base, int64_t pitch, Row row) {
        const S* s = static_cast<const S*>(base);
        ld = pitch;
        const int tid = threadIdx.x;
        if constexpr (KC) {
            constexpr int C = AStep / V;  // pieces of a row
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = s + row((tid + i * AThreads) / C) * ld + (tid % C) * V;
        } else {
            const int c = tid % (R / 4) * 4, k0 = tid / (R / 4) * F;
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = s + k0 * ld + row(c + i);
            split = p[3] != p[0] + 3;
        }
    }
    // Elements k0 .. k0 + 31; TAIL: those from K on are zeros.
    template <bool TAIL>
    __device__ __forceinline__ void fetch(int64_t k0, int64_t K) {
        const int tid = threadIdx.x;
        if constexpr (KC) {
            const int64_t left = K - k0 - (tid % (AStep / V)) * V;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!TAIL || left >= V) {
                    v[i] = *reinterpret_cast<const Pack<S, V>*>(p[i] + k0);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i].v[e] = e < left ? p[i][k0 + e] : S(0);
                }
            }
        } else {
            const int64_t left = K - k0 - tid / (R / 4) * F;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (TAIL && i >= left) {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i].v[e] = S(0);
                } else if (!split) {
                    v[i] = *reinterpret_cast<const Pack<S, V>*>(p[0] + (k0 + i) * ld);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i].v[e] = p[e][(k0 + i) * ld];
                }
            }
        }
    }
    __device__ __forceinline__ void store(char* lds) const {
        const int tid = threadIdx.x;
        constexpr int P = kParts<T>;
        if constexpr (KC) {
            constexpr int C = AStep / V;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint32_t w[P][V / 2];
                parts_of<T, V>(v[i].v, w);
                char* at = lds + (tid + i * AThreads) / C * APitch + tid % C * V * 2;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    if constexpr (V == 8)
                        *reinterpret_cast<u32x4*>(at + q * PLANE) = u32x4{w[q][0], w[q][1], w[q][2], w[q][3]};
                    else
                        *reinterpret_cast<u32x2*>(at + q * PLANE) = u32x2{w[q][0], w[q][1]};
                }
            }
        } else {
            const int c = tid % (R / 4) * 4, k0 = tid / (R / 4) * F;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S col[F];
#pragma unroll
                for (int i = 0; i < F; ++i) col[i] = v[i].v[e];
                uint32_t w[P][F / 2];
                parts_of<T, F>(col, w);
                char* at = lds + (c + e) * APitch + k0 * 2;
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    if constexpr (F == 4)
                        *reinterpret_cast<u32x2*>(at + q * PLANE) = u32x2{w[q][0], w[q][1]};
                    else
                        *reinterpret_cast<uint32_t*>(at + q * PLANE) = w[q][0];
                }
            }
        }
    }
};

// A plain product's output.
template <class T>
struct PlainOut {
    using E = T;
    static constexpr bool kGated = false;
    const FfnArgs& a;
    __device__ __forceinline__ void one(int64_t row, int64_t col, f32x4 v) const {
        const int valid = (int)(a.n - col < 4 ? a.n - col : 4);
        if (valid <= 0) return;
        const float y[4] = {v[0], v[1], v[2], v[3]};
        Quad<T>::store(static_cast<typename T::store_t*>(a.y) + row * a.ldy + col, valid, y);
    }
};

template <class Out, int F, bool AK, bool BK>
__global__ __launch_bounds__(AThreads, 2) void ffn_tile(TileArgs t, FfnArgs o) {
    using T = typename Out::E;
    using M = MmaOf<T>;
    constexpr bool G = Out::kGated;
    constexpr int P = kParts<T>, R = 32 * F, WT = 16 * F;
    constexpr int RO = G ? R / 2 : R;            // outputs of a tile
    constexpr int BUF = P == 3 && F == 4 ? 1 : 2;  // LDS buffers: one lets two blocks share a CU
    using OA = TileOperand<T, F, AK>;
    using OB = TileOperand<T, F, BK>;
    __shared__ __attribute__((aligned(16))) char lds[BUF][P * (OA::PLANE + OB::PLANE)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave >> 1, wn = wave & 1, lr = lane & 15, lq = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / t.tiles_n) * R, n0 = (int64_t)(blockIdx.x % t.tiles_n) * RO;
    OA a;
    OB b;
    a.init(t.a, t.lda, [&](int r) { return m0 + r < t.m ? m0 + r : t.m - 1; });
    b.init(t.b, t.ldb, [&](int r) {
        // Gated: each wave column's rows are half gate, half up projection.
        const int64_t col = n0 + (G ? (r / WT) * (WT / 2) + r % (WT / 2) : r);
        return (col < t.n ? col : t.n - 1) + (G && r % WT >= WT / 2 ? t.n : 0);
    });
    f32x4 acc[F][F], low[P == 3 ? F : 1][P == 3 ? F : 1];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (P == 3) low[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    auto fetch = [&](int64_t k0) {
        if (k0 + AStep <= t.k) {
            a.template fetch<false>(k0, t.k);
            b.template fetch<false>(k0, t.k);
        } else {
            a.template fetch<true>(k0, t.k);
            b.template fetch<true>(k0, t.k);
        }
    };
    auto store = [&](int buf) {
        a.store(lds[buf]);
        b.store(lds[buf] + P * OA::PLANE);
    };
    auto frag = [&](const char* plane, int row0) {
        return *reinterpret_cast<const u32x4*>(plane + (row0 + lr) * APitch + lq * 16);
    };
    fetch(0);
    store(0);
    __syncthreads();
    for (int64_t k0 = 0; k0 < t.k; k0 += AStep) {
        const int cur = BUF == 2 ? (int)((k0 / AStep) & 1) : 0;
        const bool more = k0 + AStep < t.k;
        if (more) fetch(k0 + AStep);
        const char* la = lds[cur];
        const char* lb = lds[cur] + P * OA::PLANE;
        u32x4 fa[P][F];
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
            for (int i = 0; i < F; ++i) fa[q][i] = frag(la + q * OA::PLANE, wm * WT + i * 16);
#pragma unroll
        for (int j = 0; j < F; ++j) {
            u32x4 fb[P];
#pragma unroll
            for (int q = 0; q < P; ++q) fb[q] = frag(lb + q * OB::PLANE, wn * WT + j * 16);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                if constexpr (P == 3) {
                    low[i][j] = step_mma<M>(fb[2], fa[0][i], low[i][j]);
                    low[i][j] = step_mma<M>(fb[0], fa[2][i], low[i][j]);
                    low[i][j] = step_mma<M>(fb[1], fa[1][i], low[i][j]);
                    low[i][j] = step_mma<M>(fb[1], fa[0][i], low[i][j]);
                    low[i][j] = step_mma<M>(fb[0], fa[1][i], low[i][j]);
                }
                acc[i][j] = step_mma<M>(fb[0], fa[0][i], acc[i][j]);
            }
        }
        if (BUF == 1) __syncthreads();  // read by every wave
        if (more) store(BUF == 2 ? cur ^ 1 : 0);
        __syncthreads();
    }
    const Out out{o};
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t row = m0 + wm * WT + i * 16 + lr;
        if (row >= t.m) continue;
        if constexpr (P == 3) {
#pragma unroll
            for (int j = 0; j < F; ++j) acc[i][j] += low[i][j];
        }
        if constexpr (G) {
#pragma unroll
            for (int j = 0; j < F / 2; ++j)
                out.pair(row, n0 + wn * (WT / 2) + j * 16 + 4 * lq, acc[i][j], acc[i][j + F / 2]);
        } else {
#pragma unroll
            for (int j = 0; j < F; ++j) out.one(row, n0 + wn * WT + j * 16 + 4 * lq, acc[i][j]);
        }
    }
}

// 128 x 128 tiles when they give every CU two blocks, else 64 x 64.
template <class Out, bool AK, bool BK>
hipError_t run_ffn_tile(TileArgs t, const FfnArgs& o, hipStream_t s) {
    const int64_t outs = Out::kGated ? 2 * t.n : t.n;
    const bool big = ((t.m + 127) / 128) * ((outs + 127) / 128) >= 512;
    const int64_t edge = big ? 128 : 64, ro = Out::kGated ? edge / 2 : edge;
    t.tiles_n = (int32_t)((t.n + ro - 1) / ro);
    const unsigned grid = (unsigned)((t.m + edge - 1) / edge * t.tiles_n);
    const void* fn = big ? reinterpret_cast<const void*>(&ffn_tile<Out, 4, AK, BK>)
                         : reinterpret_cast<const void*>(&ffn_tile<Out, 2, AK, BK>);
    void* args[] = {&t, const_cast<FfnArgs*>(&o)};
    return hipLaunchKernel(fn, dim3(grid), dim3(AThreads), args, 0, s);
}

// The products with the rows of W, from a product's own arguments.
template <class Out>
hipError_t run_ffn_tile(const FfnArgs& a, hipStream_t s) {
    constexpr int es = sizeof(typename Out::E::store_t);
    return run_ffn_tile<Out, true, true>(TileArgs{a.x, a.w, a.m, a.n, a.k, a.ldx / es, a.ldw / es, 0}, a, s);
}

}  // namespace mmk
