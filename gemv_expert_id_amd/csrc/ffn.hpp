// Pieces shared by the feed-forward products (gated.hip, i8.hip): operand
// types, one 64-byte step of 16 x 16 matrix instructions, and what becomes of a
// lane's four neighbouring sums.
//
// Types are handled by their bytes: a fragment is 16 rows of 64 bytes, lane l
// holding the 16 bytes at chunk l / 16 of row l % 16, in both operands; f16 and bf16
// take one 16x16x32 instruction for it, 8-bit codes one 16x16x64. (The order of the
// contraction inside a step is free as long as both operands share it.)
#pragma once

#include <type_traits>

#include "common.hpp"
#include "gate.hpp"
#include "kernels.hpp"

namespace mmk {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

struct TI8 {
    using store_t = int8_t;
    static constexpr int code = 3;
    static constexpr int Elems16 = 16;
};

template <class E> struct AccOf { using type = f32x4; };
template <> struct AccOf<TI8> { using type = i32x4; };

template <class E>
__device__ __forceinline__ typename AccOf<E>::type step_mma(u32x4 w, u32x4 x, typename AccOf<E>::type acc) {
    if constexpr (E::code == 1) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, w), __builtin_bit_cast(f16x8, x),
                                                      acc, 0, 0, 0);
    } else if constexpr (E::code == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x),
                                                       acc, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x),
                                                     acc, 0, 0, 0);
    }
}

// Transposing LDS read (ds_read_b64_tr_b16): in each group of 16 lanes, lane j gets
// element j % 4 of the four 16-bit elements at the addresses of lanes j / 4, j / 4 + 4,
// j / 4 + 8 and j / 4 + 12.
__device__ __forceinline__ u32x2 read_transposed(const char* p) {
    typedef short v4i16 __attribute__((ext_vector_type(4)));
    const v4i16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16*)(const_cast<char*>(p)));
    return __builtin_bit_cast(u32x2, v);
}

// Up to four neighbouring elements of a row: whole at an aligned address, one
// by one at others and at the row's end.
template <class T>
struct Quad {
    using S = typename T::store_t;
    static constexpr uintptr_t kMask = 4 * sizeof(S) - 1;

    static __device__ __forceinline__ void load(const S* p, int valid, float (&v)[4]) {
        if (valid >= 4 && (reinterpret_cast<uintptr_t>(p) & kMask) == 0) {
            if constexpr (sizeof(S) == 4) {
                const f32x4 q = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = q[i];
            } else {
                const u32x2 q = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = widen(T{}, (uint16_t)(q[i / 2] >> (16 * (i % 2))));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i < valid ? widen(T{}, p[i]) : 0.f;
        }
    }
    static __device__ __forceinline__ void store(S* p, int valid, const float (&v)[4]) {
        if (valid >= 4 && (reinterpret_cast<uintptr_t>(p) & kMask) == 0) {
            if constexpr (sizeof(S) == 4) {
                *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
            } else {
                u32x2 q;
                q[0] = (uint32_t)narrow(T{}, v[0]) | ((uint32_t)narrow(T{}, v[1]) << 16);
                q[1] = (uint32_t)narrow(T{}, v[2]) | ((uint32_t)narrow(T{}, v[3]) << 16);
                *reinterpret_cast<u32x2*>(p) = q;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < valid) p[i] = narrow(T{}, v[i]);
        }
    }
};

// What a product does with the sums of token `row`, outputs col .. col + 3: pair()
// takes a gate's and an up projection's, one() a plain product's. Columns from n
// on are not stored. Each is rounded to the output type once.
//
// h = act(g) * u from the f32 sums, and the sums themselves where they are kept.
template <class T>
struct GatedOut {
    using E = T;
    static constexpr bool kGated = true;
    const FfnArgs& a;
    template <class A>
    __device__ __forceinline__ void pair(int64_t row, int64_t col, A g, A u) const {
        using S = typename T::store_t;
        const int valid = (int)(a.n - col < 4 ? a.n - col : 4);
        if (valid <= 0) return;
        float h[4], gs[4], us[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gs[i] = g[i];
            us[i] = u[i];
            h[i] = gate_act(a.gate, gs[i]) * us[i];
        }
        Quad<T>::store(static_cast<S*>(a.y) + row * a.ldy + col, valid, h);
        if (a.pre_w) {
            S* p = static_cast<S*>(a.pre_w) + row * a.ldpre + col;
            Quad<T>::store(p, valid, gs);
            Quad<T>::store(p + a.n, valid, us);
        }
    }
};

// Gradients of the pre-activations from the f32 sums, which are not kept.
template <class T>
struct GradOut {
    using E = T;
    static constexpr bool kGated = true;
    const FfnArgs& a;
    template <class A>
    __device__ __forceinline__ void pair(int64_t row, int64_t col, A g, A u) const {
        using S = typename T::store_t;
        const int valid = (int)(a.n - col < 4 ? a.n - col : 4);
        if (valid <= 0) return;
        float d[4], dg[4], du[4];
        Quad<T>::load(static_cast<const S*>(a.dh) + row * a.ldy + col, valid, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) gate_grad(a.gate, g[i], u[i], d[i], &dg[i], &du[i]);
        S* p = static_cast<S*>(a.pre_w) + row * a.ldpre + col;
        Quad<T>::store(p, valid, dg);
        Quad<T>::store(p + a.n, valid, du);
    }
};

// Whole sums of codes, rounded to f32, times the channel's scale, then the token's:
// three roundings of 2^-24 before the gate or the output's own.
template <class T, bool GATED>
struct CodesOut {
    using E = TI8;
    static constexpr bool kGated = GATED;
    const FfnArgs& a;
    __device__ __forceinline__ float scaled(int32_t sum, float channel, float token) const {
        return (float)sum * channel * token;
    }
    template <class A>
    __device__ __forceinline__ void pair(int64_t row, int64_t col, A g, A u) const {
        const int valid = (int)(a.n - col < 4 ? a.n - col : 4);
        if (valid <= 0) return;
        const float token = a.sx[row];
        float sg[4], su[4], y[4];
        Quad<TF32>::load(a.sw + col, valid, sg);
        Quad<TF32>::load(a.sw + a.n + col, valid, su);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = gate_act(a.gate, scaled(g[i], sg[i], token)) * scaled(u[i], su[i], token);
        Quad<T>::store(static_cast<typename T::store_t*>(a.y) + row * a.ldy + col, valid, y);
    }
    template <class A>
    __device__ __forceinline__ void one(int64_t row, int64_t col, A v) const {
        const int valid = (int)(a.n - col < 4 ? a.n - col : 4);
        if (valid <= 0) return;
        const float token = a.sx[row];
        float s[4], y[4];
        Quad<TF32>::load(a.sw + col, valid, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = scaled(v[i], s[i], token);
        Quad<T>::store(static_cast<typename T::store_t*>(a.y) + row * a.ldy + col, valid, y);
    }
};

}  // namespace mmk
