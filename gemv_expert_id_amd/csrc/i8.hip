// Rows to 8-bit codes with a scale each, and products of codes (mm.h,
// "Feed-forward block").
#include "ffn_pipe.hpp"

namespace mmk {

namespace {

// Largest magnitude as bits that compare like it, NaN above infinity; 16-bit
// elements two at a time.
template <class T>
__device__ __forceinline__ uint32_t top_of(u32x4 v, uint32_t top) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T::code == 0) {
            const uint32_t m = v[i] & 0x7fffffffu;
            top = m > top ? m : top;
        } else {
            top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu),
                                                                         __builtin_bit_cast(u16x2, top)));
        }
    }
    return top;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A row's scale from its largest magnitude, and whether the row is finite.
template <class T>
__device__ __forceinline__ bool row_scale(uint32_t top, float* s) {
    float amax;
    if constexpr (T::code == 0) amax = __uint_as_float(top);
    else amax = widen(T{}, (uint16_t)top);
    const bool finite = amax < __builtin_inff();
    const float q = amax / 127.f;
    *s = finite && q < 0x1p-126f ? 0x1p-126f : q;
    return finite;
}

// x / s to the nearest whole number, ties to even, exactly. The quotient by
// reciprocal picks a number at most one off; the remainder x - q s is a multiple of
// half a step of s no larger than s, so f32 holds it and its comparison with s / 2
// decides. (1.5 * 2^23 added and taken back rounds to a whole number.)
constexpr float kMagic = 12582912.f;
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    float q = __builtin_fmaf(x, inv, kMagic) - kMagic;
    const float r = __builtin_fmaf(-q, s, x), h = 0.5f * s;
    const int odd = (int)q & 1;
    if (r > h || (r == h && odd)) q += 1.f;
    else if (r < -h || (r == -h && odd)) q -= 1.f;
    return (int)q;
}

// Codes of one 16-byte piece, four to a register. The quotient by reciprocal is off
// by less than 2^-15, so it decides unless an element lies within 2^-14 of a half;
// one wave in fifteen finds such an element and takes the exact form.
template <class T>
__device__ __forceinline__ void codes_of(u32x4 v, float s, float inv, uint32_t (&out)[T::Elems16 / 4]) {
    constexpr int V = T::Elems16;
    float x[V];
    if constexpr (V == 4) unpack4(v, x);
    else unpack8(T{}, v, x);
    uint32_t bits[V];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float r = __builtin_fmaf(x[i], inv, kMagic);
        off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(x[i], inv, kMagic - r)));
        bits[i] = __float_as_uint(r);
    }
    if (off > 0.5f - 0x1p-14f) {
#pragma unroll
        for (int i = 0; i < V; ++i) bits[i] = (uint32_t)code_of(x[i], s, inv);
    }
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(bits[4 * i + 1], bits[4 * i], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(bits[4 * i + 3], bits[4 * i + 2], 0x04000c0cu);
        out[i] = lo | hi;
    }
}

// W waves a row (4 rows of one wave each in a block, or one row in a block), the row
// in registers as NC pieces of 16 bytes a lane: read once. NC == 0: a longer row,
// read twice. Bound by memory: 8191 x 11008 bf16 in 52 us, 5.2 TB/s.
template <class T, int W, int NC>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void i8_quant(QuantArgs a) {
    using S = typename T::store_t;
    constexpr int V = T::Elems16, LANES = 64 * W, WB = W == 1 ? 4 : W;
    using In = Pack<S, V>;
    using Codes = Pack<int8_t, V>;
    __shared__ uint32_t tops[W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int at = W == 1 ? lane : (int)threadIdx.x;
    const int64_t pieces = (a.k + V - 1) / V;
    for (int64_t i = W == 1 ? (int64_t)blockIdx.x * WB + wave : (int64_t)blockIdx.x; i < a.m;
         i += (int64_t)gridDim.x * (W == 1 ? WB : 1)) {
        const S* x = static_cast<const S*>(a.x) + i * a.ldx;
        int8_t* q = a.q + i * a.ldq;
        auto load = [&](int64_t c) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if ((c + 1) * V <= a.k) {
                v = __builtin_bit_cast(u32x4, *reinterpret_cast<const In*>(x + c * V));
            } else if (c < pieces) {
                for (int e = 0; e < V && c * V + e < a.k; ++e) {
                    if constexpr (V == 4) v[e] = __float_as_uint(x[c * V + e]);
                    else v[e / 2] |= (uint32_t)x[c * V + e] << (16 * (e % 2));
                }
            }
            return v;
        };
        auto store = [&](int64_t c, const uint32_t (&w)[V / 4]) {
            if ((c + 1) * V <= a.k) {
                *reinterpret_cast<Codes*>(q + c * V) = *reinterpret_cast<const Codes*>(w);
            } else if (c < pieces) {
                for (int e = 0; e < V && c * V + e < a.k; ++e) q[c * V + e] = (int8_t)(w[e / 4] >> (8 * (e % 4)));
            }
        };
        u32x4 v[NC ? NC : 1];
        uint32_t top = 0;
        if constexpr (NC > 0) {
#pragma unroll
            for (int u = 0; u < NC; ++u) v[u] = load(at + u * LANES);
#pragma unroll
            for (int u = 0; u < NC; ++u) top = top_of<T>(v[u], top);
        } else {
            for (int64_t c = at; c < pieces; c += LANES) top = top_of<T>(load(c), top);
        }
        if constexpr (V == 8) top = larger(top >> 16, top & 0xffffu);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = larger(top, __shfl_xor(top, o, kWave));
        if constexpr (W > 1) {
            if (lane == 0) tops[wave] = top;
            __syncthreads();
#pragma unroll
            for (int u = 0; u < W; ++u) top = larger(top, tops[u]);
            __syncthreads();  // read before the next row's
        }
        float s;
        const bool finite = row_scale<T>(top, &s);
        if (at == 0) a.scales[i] = s;
        const float inv = finite ? 1.f / s : 0.f;
        auto put = [&](int64_t c, u32x4 piece) {
            uint32_t w[V / 4] = {};
            if (finite) codes_of<T>(piece, s, inv, w);
            store(c, w);
        };
        if constexpr (NC > 0) {
#pragma unroll
            for (int u = 0; u < NC; ++u)
                if (at + u * LANES < pieces) put(at + u * LANES, v[u]);
        } else {
            for (int64_t c = at; c < pieces; c += LANES) put(c, load(c));
        }
    }
}

template <class T>
hipError_t run_quant(const QuantArgs& a, hipStream_t s) {
    const int64_t pieces = (a.k + T::Elems16 - 1) / T::Elems16;
    const int64_t cap = 1 << 20;
    void* args[] = {const_cast<QuantArgs*>(&a)};
#define MM_QUANT(W, NC)                                                                                          \
    if (pieces <= 64 * W * NC)                                                                                   \
        return hipLaunchKernel(reinterpret_cast<const void*>(&i8_quant<T, W, NC>),                               \
                               dim3((unsigned)(W == 1 ? ((a.m + 3) / 4 < cap ? (a.m + 3) / 4 : cap)              \
                                                      : (a.m < cap ? a.m : cap))),                               \
                               dim3(W == 1 ? 256 : 64 * W), args, 0, s);
    if (a.m >= 1024) {
        MM_QUANT(1, 1) MM_QUANT(1, 2) MM_QUANT(1, 4) MM_QUANT(4, 2) MM_QUANT(4, 4) MM_QUANT(4, 6) MM_QUANT(4, 8)
    }
    MM_QUANT(1, 1) MM_QUANT(4, 1) MM_QUANT(4, 2) MM_QUANT(16, 1) MM_QUANT(16, 2) MM_QUANT(16, 4) MM_QUANT(16, 8)
#undef MM_QUANT
    return hipLaunchKernel(reinterpret_cast<const void*>(&i8_quant<T, 16, 0>), dim3((unsigned)(a.m < cap ? a.m : cap)),
                           dim3(1024), args, 0, s);
}

template <class T>
hipError_t run_i8(const FfnArgs& a, hipStream_t s, Launched* L) {
    return a.gate ? run_ffn<CodesOut<T, true>>(a, s, L) : run_ffn<CodesOut<T, false>>(a, s, L);
}

}  // namespace

hipError_t launch_i8_quant(const QuantArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_I8_QUANT;
    return a.dtype == 0 ? run_quant<TF32>(a, s) : a.dtype == 1 ? run_quant<TF16>(a, s) : run_quant<TBF16>(a, s);
}

hipError_t launch_i8(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_I8;
    return a.dtype == 0 ? run_i8<TF32>(a, s, L) : a.dtype == 1 ? run_i8<TF16>(a, s, L) : run_i8<TBF16>(a, s, L);
}

}  // namespace mmk
