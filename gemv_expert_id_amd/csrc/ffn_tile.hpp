// Tiled products of the feed-forward block for f32, and for 16-bit rows of any
// alignment: C[i][j] = sum_p A(i, p) B(j, p), each operand with p contiguous
// (element (i, p) at i * ld + p) or strided (at p * ld + i).
//
// f32 operands enter the matrix instructions as three bf16 parts (8 + 8 + 8 bits,
// exact down to 2^-133) and six products of parts, 00 01 10 11 02 20. What is left out,
// 12 21 22, is below 2^-21 of a product, 0.7 2^-24 in the mean, and always towards zero:
// parts are cut, not rounded, so that none of the largest numbers becomes an infinity.
// 16x16x32 bf16 takes 16 cycles, f32 instructions 256 for the same tile: 96 for the six.
// The products of upper parts have an accumulator of their own, so the small ones are not
// rounded away. Operands with bits below 2^-133 (any below 2^-110) are noticed while they
// are parted; their sums, and those with infinities, are computed again by f32
// instructions (f32_join). 16-bit operands are one part.
//
// A group of 4 waves (2 x 2) computes a tile of 32 FM x 32 FN, each wave SUB steps of
// 32 elements of k an iteration; a block has KS groups, which take different steps
// and are joined through LDS at the end (few tiles: more loads in flight). Operands
// are staged through registers: the next iteration's are fetched before the current
// one is multiplied, in 16-byte pieces at any address, along k or along the rows. LDS
// keeps a contiguous operand by rows, padded by 16 bytes so that the 16 rows of a
// fragment read start in distinct banks, and a strided one by k, as it comes; its
// fragments take two transposing reads each. Rows past the end repeat others (their
// sums are not stored); elements of k past the end are zeros in both operands. A piece
// that passes an end is fetched from where it still lies inside and moved up in
// registers, so that edges cost no loads of single elements.
//
// Large f32 products: 4096 x 8192 over 4096 takes 1430 us, 192 TFLOP/s, 1150 of bf16
// products. Matrix units are busy for 54% of the cycles, vector instructions issue in 46%,
// LDS conflicts take 27%; the 128 x 128 tile holds 256 registers and spills 35 more. Rows
// of 16 bits that no pipelined form takes are bound by the staging through registers
// (2000 x 4100 over 10000 bf16 344 us, 477 TFLOP/s).
#pragma once

#include "ffn.hpp"

namespace mmk {

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

constexpr uint32_t kUpperHalves = 0x07060302u;  // (v_perm_b32) of two registers

// N elements as their parts, two to a register. `lost` collects what the first two
// parts leave: the third one holds it unless some of its lower 16 bits are set
// (parts_lost), as only bits of f32 below 2^-133 are. (One instruction in 12. In
// assembly that the third part passes through, or the compiler would gather the
// remainders until later and spill: 160 x 11008 x 4096 in 650 us instead of 287.)
template <class T, int N>
__device__ __forceinline__ void parts_of(const typename T::store_t (&e)[N], uint32_t (&out)[kParts<T>][N / 2],
                                         uint32_t& lost) {
    if constexpr (T::code == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float lo = e[2 * i], hi = e[2 * i + 1];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                out[q][i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), kUpperHalves);
                lo -= __uint_as_float(__float_as_uint(lo) & 0xFFFF0000u);
                hi -= __uint_as_float(__float_as_uint(hi) & 0xFFFF0000u);
            }
            out[2][i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), kUpperHalves);
            asm("v_or3_b32 %0, %2, %3, %0" : "+&v"(lost), "+v"(out[2][i]) : "v"(lo), "v"(hi));
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[0][i] = (uint32_t)e[2 * i] | ((uint32_t)e[2 * i + 1] << 16);
    }
}

__device__ __forceinline__ bool parts_lost(uint32_t lost) { return (lost & 0xFFFFu) != 0; }

// Elements 4 g .. 4 g + 3 and 16 + 4 g .. of a step of 32 of a row (`row` at its element
// 4 g, g = lane / 16 % 4), C contiguous or `stride` apart; with TAIL, zeros from `valid` on.
template <bool C, bool TAIL>
__device__ __forceinline__ void row_eight(const float* row, int64_t stride, int valid, float (&v)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (C && !TAIL) {
            const Pack<float, 4> four = *reinterpret_cast<const Pack<float, 4>*>(row + 16 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = four.v[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = !TAIL || 16 * h + e < valid ? row[(16 * h + e) * (C ? 1 : stride)] : 0.f;
        }
    }
}

// The sums of a wave's FM x FN fragments, in acc, from those of upper parts and of the small
// products; by f32 instructions straight from memory where parts do not give them:
// - An infinity leaves NaN in the small products.
// - `lost` says that parts of some rows lack bits; a look at the rows finds them. What is
//   lost of k products is less than k 2^-133 (|x| + |w|), with the largest magnitudes of the
//   two rows, and changes nothing in a sum 2^24 times as large. (A few tiny values among
//   ordinary ones, as gradients behind a gate that is almost shut, cost the look, 1.7 to 4
//   times the product; rows of tiny values take 2.5 to 6.5 times as long.) A NaN may be an
//   infinity times a lost value.
// Each sum goes by its own rows: what others of the wave hold does not change it, and
// neighbouring tiles that both store a sum store the same.
//
// `x(lr, i)` and `w(lr, j)` point to element 0 of row lr of a fragment, whose elements lie
// together (XC, WC) or xs (ws) apart; the wave takes every KS-th step of 32 elements from
// step kg on. Instruction q of 16 elements takes element 4 g + q of lanes 16 g on, in both
// operands. (The lane is hidden from the compiler, which would otherwise hold the addresses
// in registers all through the loop before.)
template <int KS, bool XC, bool WC, int FM, int FN, class X, class W>
__device__ __forceinline__ void f32_join(int64_t k, int kg, bool lost, X x, int64_t xs, W w, int64_t ws, f32x4 (&acc)[FM][FN],
                                         const f32x4 (&low)[FM][FN]) {
    uint64_t again = 0;  // the sums to compute, element e of fragment (i, j) at 4 (i FN + j) + e
    bool nan = false;
#pragma unroll
    for (int f = 0; f < FM * FN * 4; ++f) nan |= __builtin_isnan(low[f / 4 / FN][f / 4 % FN][f % 4]);
    if (__any(nan)) {
#pragma unroll
        for (int f = 0; f < FM * FN * 4; ++f)
            if (__builtin_isnan(low[f / 4 / FN][f / 4 % FN][f % 4]) && __builtin_isinf(acc[f / 4 / FN][f / 4 % FN][f % 4]))
                again |= 1ull << f;
    }
#pragma unroll
    for (int f = 0; f < FM * FN; ++f) acc[f / FN][f % FN] += low[f / FN][f % FN];
    if (!__any(lost || again)) return;
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int lr = lane & 15, lq = lane >> 4;
    const int64_t first = kg * 32 + 4 * lq, whole = k / 32, end = whole * 32;
    const bool tail = k % 32 && whole % KS == kg;
    const int valid = (int)(k - end) - 4 * lq;
    // Largest magnitude of a row, and which of the 16 rows (bit lr) hold bits below 2^-133:
    // numbers below 2^-110 that are no multiple of it.
    struct Row {
        float top;
        uint32_t lack;
    };
    const auto look = [&](const float* row, int64_t stride, auto C_) {
        constexpr bool C = decltype(C_)::value;
        float top = 0.f, v[8];
        bool lack = false;
        const auto take = [&] {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = __builtin_fabsf(v[e]), units = a * 0x1p66f * 0x1p67f;
                top = __builtin_fmaxf(top, a);
                lack |= a < 0x1p-110f && units != __builtin_truncf(units);
            }
        };
        const float* p = row + first * (C ? 1 : stride);
#pragma unroll 4
        for (int64_t s = kg * 32; s < end; s += 32 * KS, p += 32 * KS * (C ? 1 : stride)) {
            row_eight<C, false>(p, stride, 0, v);
            take();
        }
        if (tail) {
            row_eight<C, true>(row + (end + 4 * lq) * (C ? 1 : stride), stride, valid, v);
            take();
        }
        top = __builtin_fmaxf(top, __shfl_xor(top, 16, kWave));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32, kWave));
        const uint64_t all = __ballot(lack);
        const uint32_t half = (uint32_t)(all | all >> 32);
        return Row{top, (half | half >> 16) & 0xFFFFu};
    };
    if (__any(lost)) {
        const float least = (float)k * 0x1p-109f;
        Row rx[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) rx[i] = look(x(lr, i), xs, std::bool_constant<XC>{});
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const Row rw = look(w(lr, j), ws, std::bool_constant<WC>{});
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 4 * lq + e;  // the row of sum e
                const float up = __shfl(rw.top, r, kWave);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    if (((rx[i].lack >> lr | rw.lack >> r) & 1) && rx[i].top > 0.f && up > 0.f &&
                        !(__builtin_fabsf(acc[i][j][e]) >= least * (rx[i].top + up)))
                        again |= 1ull << (4 * (i * FN + j) + e);
            }
        }
        if (!__any(again != 0)) return;
    }
    constexpr int JN = FN % 2 ? 1 : 2;  // fragments of w at a time
#pragma unroll
    for (int j = 0; j < FN; j += JN) {
        const float* px[FM];
        const float* pw[JN];
        f32x4 sum[FM][JN];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            px[i] = x(lr, i) + first * (XC ? 1 : xs);
#pragma unroll
            for (int u = 0; u < JN; ++u) sum[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int u = 0; u < JN; ++u) pw[u] = w(lr, j + u) + first * (WC ? 1 : ws);
        const auto step = [&](auto tail_) {
            constexpr bool TAIL = decltype(tail_)::value;
            float fx[FM][8], fw[JN][8];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                row_eight<XC, TAIL>(px[i], xs, valid, fx[i]);
                px[i] += 32 * KS * (XC ? 1 : xs);
            }
#pragma unroll
            for (int u = 0; u < JN; ++u) {
                row_eight<WC, TAIL>(pw[u], ws, valid, fw[u]);
                pw[u] += 32 * KS * (WC ? 1 : ws);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int u = 0; u < JN; ++u)
                        sum[i][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(fw[u][q], fx[i][q], sum[i][u], 0, 0, 0);
        };
#pragma unroll 1
        for (int64_t s = kg * 32; s < end; s += 32 * KS) step(std::false_type{});
        if (tail) step(std::true_type{});
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int u = 0; u < JN; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (again >> (4 * (i * FN + j + u) + e) & 1) acc[i][j + u][e] = sum[i][u][e];
    }
}

// One operand's share of a thread: R rows by KT elements of k, spread over NT threads.
template <class T, int R, int KT, int NT, bool KC>
struct TileOperand {
    using S = typename T::store_t;
    static constexpr int P = kParts<T>;
    static constexpr int V = T::Elems16;                     // elements of a piece
    static constexpr int PITCH = KC ? KT * 2 + 16 : R * 2;   // bytes between LDS rows (of k, strided)
    static constexpr int PLANE = KC ? R * PITCH : KT * PITCH;  // bytes of one part
    static constexpr int C = KC ? KT / V : R / V;            // pieces of a row
    static constexpr int ALL = R * KT / V;                   // pieces
    static constexpr int N = ALL > NT ? ALL / NT : 1;        // of a thread (of the first ALL, if fewer)
    static_assert(N * NT == ALL || N == 1, "whole pieces");
    static_assert(NT % C == 0, "a thread's pieces lie at one place of their rows");
    Pack<S, V> v[N];
    const S* p[KC ? N : 1];  // row starts; or the columns
    int64_t ld;
    int shift;               // a piece that passes the end is fetched this many elements earlier
    int some;                // an operand shorter than a piece: elements to fetch one by one (else 0)
    uint32_t lost = 0;       // (parts_of)

    static __device__ __forceinline__ int piece(int i) { return (int)threadIdx.x + i * NT; }
    // Place of this thread's pieces in their rows.
    static __device__ __forceinline__ int place() { return (int)threadIdx.x % C * V; }
    // Strided: 16-byte chunk swizzle of k-row r, by which the 16 k-rows of a
    // transposing read cover all banks twice.
    static __device__ __forceinline__ int swizzle(int r) {
        if constexpr (R >= 128) return 2 * ((r & 3) + 4 * ((r >> 3) & 1));
        else if constexpr (R == 64) return 2 * (((r >> 1) & 1) + 2 * ((r >> 3) & 1));
        else return 2 * ((r >> 3) & 1);
    }
    // Contiguous: `row(r)` is the operand's row that tile row r stands for, already
    // inside it. Strided: the tile's columns are first .. first + R - 1 of `cols`.
    template <class Row>
    __device__ __forceinline__ void init(const void* base, int64_t pitch, int64_t first, int64_t cols, Row row) {
        const S* s = static_cast<const S*>(base);
        ld = pitch;
        shift = some = 0;
        if constexpr (KC) {
#pragma unroll
            for (int i = 0; i < N; ++i) p[i] = s + row(piece(i) / C) * ld;
        } else {
            const int64_t c = first + place();
            const int64_t over = c + V - cols;  // elements past the end
            if (cols < V) {
                some = (int)cols;
                p[0] = s;  // (first is 0)
            } else {
                p[0] = s + (over > 0 ? cols - V : c);
                if (over > 0 && over < V) shift = (int)over;
            }
        }
    }
    // Elements k0 .. k0 + KT - 1; TAIL: those from K on are zeros.
    template <bool TAIL>
    __device__ __forceinline__ void fetch(int64_t k0, int64_t K) {
        if (ALL < NT && (int)threadIdx.x >= ALL) return;
        const int64_t at = k0 + place();
        if constexpr (KC && TAIL) {
            const int64_t over = at + V - K;
            shift = over > 0 ? (int)(over < V ? over : V) : 0;
            some = K < V ? (int)K : 0;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (KC) {
                if (!TAIL || (shift == 0 && !some)) v[i] = *reinterpret_cast<const Pack<S, V>*>(p[i] + at);
                else if (!some) v[i] = *reinterpret_cast<const Pack<S, V>*>(p[i] + K - V);
                else few(v[i], p[i], place() ? 0 : some);
            } else {
                const int64_t k = k0 + piece(i) / C;
                if (TAIL && k >= K) few(v[i], p[0], 0);
                else if (!some) v[i] = *reinterpret_cast<const Pack<S, V>*>(p[0] + k * ld);
                else few(v[i], p[0] + k * ld, place() ? 0 : some);
            }
        }
        if (KC && TAIL && some) shift = 0;
    }
    static __device__ __forceinline__ void few(Pack<S, V>& to, const S* from, int n) {
#pragma unroll
        for (int e = 0; e < V; ++e) to.v[e] = e < n ? from[e] : S(0);
    }
    __device__ __forceinline__ void store(char* lds) {
        if (ALL < NT && (int)threadIdx.x >= ALL) return;
        if (shift) {  // the elements wanted to the front, zeros behind
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int b = 1; b <= V; b *= 2)
                    if (shift & b) {
#pragma unroll
                        for (int e = 0; e < V; ++e) v[i].v[e] = e + b < V ? v[i].v[e + b < V ? e + b : 0] : S(0);
                    }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t w[P][V / 2];
            parts_of<T, V>(v[i].v, w, lost);
            const int r = piece(i) / C, at = place() * 2;
            char* to = lds + r * PITCH + (KC ? at : (((at >> 4) ^ swizzle(r)) << 4) + (at & 15));
#pragma unroll
            for (int q = 0; q < P; ++q) {
                if constexpr (V == 8)
                    *reinterpret_cast<u32x4*>(to + q * PLANE) = u32x4{w[q][0], w[q][1], w[q][2], w[q][3]};
                else
                    *reinterpret_cast<u32x2*>(to + q * PLANE) = u32x2{w[q][0], w[q][1]};
            }
        }
    }
    // The lane's eight elements of rows row0 .. row0 + 15 in step `step` (32 of k) of a
    // plane: row lane % 16, elements 8 (lane / 16) of the step on.
    static __device__ __forceinline__ u32x4 frag(const char* plane, int row0, int step) {
        const int lane = threadIdx.x & 63, g = lane >> 4, s = lane & 15;
        if constexpr (KC) {
            return *reinterpret_cast<const u32x4*>(plane + (row0 + s) * PITCH + step * 64 + g * 16);
        } else {
            // Lane s of group g addresses k-rows 8 g + s / 4 and + 4, columns 4 (s % 4) on.
            const int r0 = step * 32 + 8 * g + (s >> 2), r1 = r0 + 4, c = row0 / 8 + ((s & 3) >> 1);
            const u32x2 lo = read_transposed(plane + r0 * PITCH + ((c ^ swizzle(r0)) << 4) + 8 * (s & 1));
            const u32x2 hi = read_transposed(plane + r1 * PITCH + ((c ^ swizzle(r1)) << 4) + 8 * (s & 1));
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
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

template <class T, int FM_, int FN_, int SUB_, int KS_>
struct TileShape {
    static constexpr int FM = FM_, FN = FN_, SUB = SUB_, KS = KS_;
    static constexpr int BM = 32 * FM, BN = 32 * FN, KT = 32 * SUB * KS, THREADS = 256 * KS;
    static constexpr int BYTES = kParts<T> * (BM + BN) * (KT * 2 + 16);  // one LDS buffer, at most
    // Two buffers where a CU still holds two blocks (one, where the groups split k).
    static constexpr int BUF = 2 * BYTES * (KS > 1 ? 1 : 2) <= 160 * 1024 ? 2 : 1;
};

template <class Out, class Z, bool AK, bool BK>
__global__ __launch_bounds__(Z::THREADS, Z::KS > 1 ? Z::KS : 2) void ffn_tile(TileArgs t, FfnArgs o) {
    using T = typename Out::E;
    using M = MmaOf<T>;
    constexpr bool G = Out::kGated;
    constexpr int P = kParts<T>, FM = Z::FM, FN = Z::FN, TM = 16 * FM, TN = 16 * FN, KT = Z::KT, BUF = Z::BUF;
    constexpr int RO = G ? Z::BN / 2 : Z::BN;  // outputs of a tile
    using OA = TileOperand<T, Z::BM, KT, Z::THREADS, AK>;
    using OB = TileOperand<T, Z::BN, KT, Z::THREADS, BK>;
    static_assert(P * (OA::PLANE + OB::PLANE) <= Z::BYTES, "LDS buffer");
    extern __shared__ __attribute__((aligned(16))) char tile_lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int kg = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1, lr = lane & 15, lq = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / t.tiles_n) * Z::BM, n0 = (int64_t)(blockIdx.x % t.tiles_n) * RO;
    OA a;
    OB b;
    const auto row_a = [&](int r) { return m0 + r < t.m ? m0 + r : t.m - 1; };
    a.init(t.a, t.lda, m0, t.m, row_a);
    const auto row_b = [&](int r) {
        // Gated: each wave column's rows are half gate, half up projection.
        const int64_t col = n0 + (G ? (r / TN) * (TN / 2) + r % (TN / 2) : r);
        return (col < t.n ? col : t.n - 1) + (G && r % TN >= TN / 2 ? t.n : 0);
    };
    b.init(t.b, t.ldb, n0, t.n, row_b);
    f32x4 acc[FM][FN], low[P == 3 ? FM : 1][P == 3 ? FN : 1];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (P == 3) low[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    auto fetch = [&](int64_t k0) {
        if (k0 + KT <= t.k) {
            a.template fetch<false>(k0, t.k);
            b.template fetch<false>(k0, t.k);
        } else {
            a.template fetch<true>(k0, t.k);
            b.template fetch<true>(k0, t.k);
        }
    };
    auto store = [&](int buf) {
        a.store(tile_lds + buf * Z::BYTES);
        b.store(tile_lds + buf * Z::BYTES + P * OA::PLANE);
    };
    fetch(0);
    store(0);
    __syncthreads();
    for (int64_t k0 = 0; k0 < t.k; k0 += KT) {
        const int cur = BUF == 2 ? (int)((k0 / KT) & 1) : 0;
        const bool more = k0 + KT < t.k;
        if (more) fetch(k0 + KT);
#pragma unroll
        for (int s = 0; s < Z::SUB; ++s) {
            const char* la = tile_lds + cur * Z::BYTES;
            const char* lb = la + P * OA::PLANE;
            const int step = kg * Z::SUB + s;
            u32x4 fa[P][FM];
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int i = 0; i < FM; ++i) fa[q][i] = OA::frag(la + q * OA::PLANE, wm * TM + i * 16, step);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                u32x4 fb[P];
#pragma unroll
                for (int q = 0; q < P; ++q) fb[q] = OB::frag(lb + q * OB::PLANE, wn * TN + j * 16, step);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
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
        }
        if (BUF == 1) __syncthreads();  // read by every wave
        if (more) store(BUF == 2 ? cur ^ 1 : 0);
        __syncthreads();
    }
    if constexpr (P == 3) {
        const bool lost = __syncthreads_or(parts_lost(a.lost | b.lost));
        const auto x = [&](int r, int i) {
            return static_cast<const float*>(t.a) + row_a(wm * TM + i * 16 + r) * (AK ? t.lda : 1);
        };
        const auto w = [&](int r, int j) {
            return static_cast<const float*>(t.b) + row_b(wn * TN + j * 16 + r) * (BK ? t.ldb : 1);
        };
        f32_join<Z::KS, AK, BK>(t.k, kg, lost, x, t.lda, w, t.ldb, acc, low);
    }
    if constexpr (Z::KS > 1) {
        f32x4* part = reinterpret_cast<f32x4*>(tile_lds);
        static_assert((Z::KS - 1) * 256 * FM * FN * 16 <= Z::BUF * Z::BYTES, "partial sums fit");
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < FM * FN; ++i) part[((kg - 1) * FM * FN + i) * 256 + (threadIdx.x & 255)] = acc[i / FN][i % FN];
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int g = 1; g < Z::KS; ++g)
#pragma unroll
            for (int i = 0; i < FM * FN; ++i) acc[i / FN][i % FN] += part[((g - 1) * FM * FN + i) * 256 + threadIdx.x];
    }
    const Out out{o};
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row = m0 + wm * TM + i * 16 + lr;
        if (row >= t.m) continue;
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

template <class Out, class Z, bool AK, bool BK>
hipError_t run_tile(TileArgs t, const FfnArgs& o, hipStream_t s) {
    constexpr int RO = Out::kGated ? Z::BN / 2 : Z::BN;
    t.tiles_n = (int32_t)((t.n + RO - 1) / RO);
    const unsigned grid = (unsigned)((t.m + Z::BM - 1) / Z::BM * t.tiles_n);
    void* args[] = {&t, const_cast<FfnArgs*>(&o)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ffn_tile<Out, Z, AK, BK>), dim3(grid), dim3(Z::THREADS), args,
                           Z::BUF * Z::BYTES, s);
}

// The forms of 16-bit elements: 32 FM x 32 FN tiles, SUB steps, KS groups; and what a
// round of 512 (of 256 with four groups) costs in us, for each iteration over k and at
// its start. From 130 products of each layout in every form; the form with the lowest
// sum of rounds is within 5% of the fastest in the mean. Both sides of some borders, us:
// 3 x 3456 over 3200 bf16, two steps an iteration 14.3, one 20.5; gated 2 x 24192 over
// 2503 bf16, 48.8 and 37.1. (f32 has choices of its own: ffn_f32.hpp, ffn_strided.hpp.)
template <class Out, bool AK, bool BK>
hipError_t run_ffn_tile(const TileArgs& t, const FfnArgs& o, hipStream_t s) {
    using T = typename Out::E;
    static_assert(T::code != 0, "16 bits");
    constexpr bool ROWS = AK && BK;
    using Big = TileShape<T, 4, 4, 2, 1>;
    using Mid = TileShape<T, 2, 2, 1, 1>;
    using Deep = TileShape<T, 2, 2, 1, 4>;
    using Low = TileShape<T, 1, 2, 1, 4>;
    using Long = TileShape<T, 1, 2, 2, 4>;
    constexpr float big = ROWS ? 1.6f : 1.4f, mid = ROWS ? 0.42f : 0.36f;
    constexpr float deep = ROWS ? 1.5f : 1.36f, low = ROWS ? 0.91f : 0.96f;
    const int64_t outs = Out::kGated ? 2 * t.n : t.n;
    const auto us = [&](int bm, int bn, int kt, int at_a_time, float step, float start) {
        const int64_t tiles = ((t.m + bm - 1) / bm) * ((outs + bn - 1) / bn);
        if (bm < 128 && tiles >= (1 << 22)) return 3e38f;  // (a grid holds fewer than 2^32 threads)
        return (float)((tiles + at_a_time - 1) / at_a_time) * ((float)((t.k + kt - 1) / kt) * step + start);
    };
    if constexpr (!Out::kGated) {  // the narrowest while CUs are left
        if (((t.m + 31) / 32) * ((t.n + 31) / 32) <= 256)
            return run_tile<Out, TileShape<T, 1, 1, 2, 4>, AK, BK>(t, o, s);
    }
    const bool few = ((t.m + 31) / 32) * ((outs + 63) / 64) <= 256;
    const float b = us(128, 128, 64, 512, big, 5.f), m = us(64, 64, 32, 512, mid, 1.5f), d = us(64, 64, 128, 256, deep, 1.4f);
    const float l = few ? us(32, 64, 256, 256, 1.3f, 1.4f) : us(32, 64, 128, 256, low, 1.4f);
    if (b <= m && b <= d && b <= l) return run_tile<Out, Big, AK, BK>(t, o, s);
    if (m <= d && m <= l) return run_tile<Out, Mid, AK, BK>(t, o, s);
    if (d <= l) return run_tile<Out, Deep, AK, BK>(t, o, s);
    if (few) return run_tile<Out, Long, AK, BK>(t, o, s);
    return run_tile<Out, Low, AK, BK>(t, o, s);
}

// The products with the rows of W, from a product's own arguments.
template <class Out>
hipError_t run_ffn_tile(const FfnArgs& a, hipStream_t s) {
    constexpr int es = sizeof(typename Out::E::store_t);
    return run_ffn_tile<Out, true, true>(TileArgs{a.x, a.w, a.m, a.n, a.k, a.ldx / es, a.ldw / es, 0}, a, s);
}

}  // namespace mmk
