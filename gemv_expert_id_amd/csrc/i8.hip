// Rows to 8-bit codes with a scale each, and products of codes (mm.h,
// "Feed-forward block").
#include "ffn_pipe.hpp"

namespace mmk {

namespace {

// Magnitude of a stored value as bits that compare like it, NaN above infinity.
template <class T>
__device__ __forceinline__ uint32_t magnitude(typename T::store_t v) {
    if constexpr (T::code == 0) return __float_as_uint(v) & 0x7fffffffu;
    else return v & 0x7fffu;
}
template <class T>
__device__ __forceinline__ float from_magnitude(uint32_t bits) {
    if constexpr (T::code == 0) return __uint_as_float(bits);
    else return widen(T{}, (uint16_t)bits);
}

// x / s to the nearest whole number, ties to even, exactly. The quotient by
// reciprocal picks a number at most one off; the remainder x - q s is a multiple of
// half a step of s no larger than s, so f32 holds it and its comparison with s / 2
// decides. (1.5 * 2^23 added and taken back rounds to a whole number.)
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    constexpr float kMagic = 12582912.f;
    float q = (x * inv + kMagic) - kMagic;
    const float r = __builtin_fmaf(-q, s, x), h = 0.5f * s;
    const int odd = (int)q & 1;
    if (r > h || (r == h && odd)) q += 1.f;
    else if (r < -h || (r == -h && odd)) q -= 1.f;
    return (int)q;
}

// One block a row: the row's largest magnitude, then its codes.
template <class T>
__global__ __launch_bounds__(256) void i8_quant(QuantArgs a) {
    using S = typename T::store_t;
    __shared__ uint32_t top[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
        const S* x = static_cast<const S*>(a.x) + i * a.ldx;
        int8_t* q = a.q + i * a.ldq;
        uint32_t t = 0;
        for (int64_t p = threadIdx.x; p < a.k; p += 256) {
            const uint32_t v = magnitude<T>(x[p]);
            t = v > t ? v : t;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint32_t v = __shfl_xor(t, o, kWave);
            t = v > t ? v : t;
        }
        if (lane == 0) top[wave] = t;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 4; ++w) t = top[w] > t ? top[w] : t;
        __syncthreads();  // read before the next row's
        const float amax = from_magnitude<T>(t);
        const bool finite = amax < __builtin_inff();
        float s = amax / 127.f;
        s = finite && s < 0x1p-126f ? 0x1p-126f : s;
        if (threadIdx.x == 0) a.scales[i] = s;
        const float inv = 1.f / s;
        for (int64_t p = threadIdx.x; p < a.k; p += 256)
            q[p] = (int8_t)(finite ? code_of(widen(T{}, x[p]), s, inv) : 0);
    }
}

template <class T>
hipError_t run_i8(const FfnArgs& a, hipStream_t s, Launched* L) {
    return a.gate ? run_ffn<CodesOut<T, true>>(a, s, L) : run_ffn<CodesOut<T, false>>(a, s, L);
}

}  // namespace

hipError_t launch_i8_quant(const QuantArgs& a, hipStream_t s, Launched* L) {
    const unsigned grid = (unsigned)(a.m < (1 << 22) ? a.m : 1 << 22);
    const void* fn = a.dtype == 0   ? (const void*)&i8_quant<TF32>
                     : a.dtype == 1 ? (const void*)&i8_quant<TF16>
                                    : (const void*)&i8_quant<TBF16>;
    void* args[] = {const_cast<QuantArgs*>(&a)};
    L->kernel = MM_KERNEL_I8_QUANT;
    return hipLaunchKernel(fn, dim3(grid), dim3(256), args, 0, s);
}

hipError_t launch_i8(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_I8;
    return a.dtype == 0 ? run_i8<TF32>(a, s, L) : a.dtype == 1 ? run_i8<TF16>(a, s, L) : run_i8<TBF16>(a, s, L);
}

}  // namespace mmk
