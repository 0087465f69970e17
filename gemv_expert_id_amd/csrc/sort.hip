// Routed rows in expert order, and back to tokens: the sort's plan and its row
// gather, the weighted combination, and the gradients.
//
// Plan: a stable counting sort without scratch. Block b (one for each expert,
// and one for the rows without) counts over all ids the keys below b, which is
// the first place of its rows, and those equal to b, wave by wave; a second
// pass over the ids gives each row of b its rank. Blocks exchange nothing, and
// the ids are small next to the rows (4 bytes against a row), so reading them
// once a block costs less than a second launch or a wait between blocks.
#include "common.hpp"
#include "kernels.hpp"

namespace mmk {

namespace {

constexpr int PThreads = 1024;
constexpr int PWaves = PThreads / kWave;
constexpr int CThreads = 256;
constexpr int CWaves = CThreads / kWave;

__device__ __forceinline__ uint32_t lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

__global__ __launch_bounds__(PThreads) void sort_plan(SortArgs a) {
    __shared__ uint32_t s_less[PWaves], s_eq[PWaves];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint32_t E = a.n_experts, b = blockIdx.x;  // b == E: rows without an expert
    const int64_t R = (int64_t)a.m * a.top_k;
    // Wave w owns a contiguous piece of the routed rows.
    const int64_t piece = (R + PWaves * kWave - 1) / (PWaves * kWave) * kWave;
    const int64_t r0 = wave * piece, r1 = r0 + piece < R ? r0 + piece : R;
    uint32_t less = 0, eq = 0;
    for (int64_t r = r0 + lane; r < r1; r += kWave) {
        const uint32_t id = a.ids[r], key = id < E ? id : E;
        less += key < b;
        eq += key == b;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        less += __shfl_xor((int)less, o, kWave);
        eq += __shfl_xor((int)eq, o, kWave);
    }
    if (lane == 0) { s_less[wave] = less; s_eq[wave] = eq; }
    __syncthreads();
    uint32_t place = 0;
    for (int w = 0; w < PWaves; ++w) place += s_less[w];
    if (threadIdx.x == 0) a.offsets_w[b] = place;
    for (int w = 0; w < wave; ++w) place += s_eq[w];
    if (s_eq[wave] == 0) return;
    for (int64_t r = r0; r < r1; r += kWave) {
        const bool in = r + lane < r1;
        const uint32_t id = in ? a.ids[r + lane] : 0u, key = id < E ? id : E;
        const uint64_t mask = __ballot(in && key == b);
        if (in && key == b) {
            const uint32_t i = place + lanes_below(mask);
            a.order_w[i] = (uint32_t)(r + lane);
            a.position_w[r + lane] = i;
        }
        place += (uint32_t)__popcll(mask);
    }
}

// 16 bytes of a row that is aligned to its element only.
template <class S>
struct __attribute__((packed, aligned(sizeof(S)))) Chunk {
    u32x4 v;
};
template <class S>
__device__ __forceinline__ u32x4 ld_chunk(const S* p) {
    return reinterpret_cast<const Chunk<S>*>(p)->v;
}
template <class S>
__device__ __forceinline__ void st_chunk(S* p, u32x4 v) {
    reinterpret_cast<Chunk<S>*>(p)->v = v;
}

template <class T>
__device__ __forceinline__ void unpack(u32x4 v, float* f) {
    if constexpr (T::Elems16 == 4) unpack4(v, f);
    else unpack8(T{}, v, f);
}
template <class T>
__device__ __forceinline__ u32x4 repack(const float* f) {
    u32x4 v;
    if constexpr (T::Elems16 == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (uint32_t)narrow(T{}, f[2 * i]) | ((uint32_t)narrow(T{}, f[2 * i + 1]) << 16);
    }
    return v;
}

// xs[i] = x[order[i] / top_k], +0 past offsets[E]. The rows are moved as bits.
template <class S>
__global__ __launch_bounds__(CThreads) void sort_gather(SortArgs a) {
    constexpr int CH = 16 / sizeof(S);
    const int64_t R = (int64_t)a.m * a.top_k;
    const uint32_t live = a.offsets[a.n_experts];
    for (int64_t i = blockIdx.x; i < R; i += gridDim.x) {
        const uint32_t r = a.order[i];
        const S* src = static_cast<const S*>(a.tokens) + (int64_t)(r / a.top_k) * a.ld_tokens;
        S* dst = static_cast<S*>(a.rows_w) + i * a.ld_rows;
        const bool on = i < live && r < R;
        for (uint32_t j = threadIdx.x * CH; j < a.width; j += CThreads * CH) {
            if (j + CH <= a.width) {
                st_chunk(dst + j, on ? ld_chunk(src + j) : u32x4{0, 0, 0, 0});
            } else {
                for (uint32_t q = j; q < a.width; ++q) dst[q] = on ? src[q] : (S)0;
            }
        }
    }
}

// out[t] = residual[t] + sum_s w[t][s] y[position]; without weights each is 1.
// W: has weights. A block takes one token and one piece of its row.
template <class T, bool W>
__global__ __launch_bounds__(CThreads) void combine(SortArgs a) {
    using S = typename T::store_t;
    constexpr int CH = T::Elems16;
    const uint32_t R = a.m * a.top_k;
    const uint32_t live = a.position ? (a.offsets[a.n_experts] < R ? a.offsets[a.n_experts] : R) : R;
    const uint32_t j = (blockIdx.y * CThreads + threadIdx.x) * CH;
    if (j >= a.width) return;
    const bool whole = j + CH <= a.width;
    for (int64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        float acc[CH] = {};
        if (a.residual) {
            const S* res = static_cast<const S*>(a.residual) + t * a.ld_tokens + j;
            if (whole) unpack<T>(ld_chunk(res), acc);
            else
                for (uint32_t q = 0; j + q < a.width; ++q) acc[q] = widen(T{}, res[q]);
        }
        for (uint32_t s = 0; s < a.top_k; ++s) {
            const uint32_t r = (uint32_t)t * a.top_k + s;
            const uint32_t i = a.position ? a.position[r] : r;
            if (i >= live) continue;
            const float w = W ? a.weights[r] : 1.f;
            const S* y = static_cast<const S*>(a.rows) + (int64_t)i * a.ld_rows + j;
            float f[CH] = {};
            if (whole) unpack<T>(ld_chunk(y), f);
            else
                for (uint32_t q = 0; j + q < a.width; ++q) f[q] = widen(T{}, y[q]);
#pragma unroll
            for (int q = 0; q < CH; ++q) acc[q] = __builtin_fmaf(w, f[q], acc[q]);
        }
        S* out = static_cast<S*>(a.tokens_w) + t * a.ld_tokens + j;
        if (whole) st_chunk(out, repack<T>(acc));
        else
            for (uint32_t q = 0; j + q < a.width; ++q) out[q] = narrow(T{}, acc[q]);
    }
}

// dy[i] = w dout[t], dw = <dout[t], y[i]>. One wave for each routed row.
template <class T>
__global__ __launch_bounds__(CThreads) void combine_grad(SortArgs a) {
    using S = typename T::store_t;
    constexpr int CH = T::Elems16;
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t R = a.m * a.top_k;
    const uint32_t live = a.position ? a.offsets[a.n_experts] : R;
    for (int64_t r = (int64_t)blockIdx.x * CWaves + threadIdx.x / kWave; r < R;
         r += (int64_t)gridDim.x * CWaves) {
        const uint32_t i = a.position ? a.position[r] : (uint32_t)r;
        const bool on = i < live;
        const float w = on ? a.weights[r] : 0.f;
        const S* d = static_cast<const S*>(a.tokens) + (r / a.top_k) * a.ld_tokens;
        const S* y = static_cast<const S*>(a.rows) + (int64_t)i * a.ld_rows;
        S* dy = static_cast<S*>(a.rows_w) + (int64_t)i * a.ld_rows;
        float dot = 0.f;
        if (i < R) {
            for (uint32_t j = lane * CH; j < a.width; j += kWave * CH) {
                float g[CH] = {}, f[CH] = {}, o[CH] = {};
                if (j + CH <= a.width) {
                    if (on) {
                        unpack<T>(ld_chunk(d + j), g);
                        unpack<T>(ld_chunk(y + j), f);
                    }
#pragma unroll
                    for (int q = 0; q < CH; ++q) {
                        dot = __builtin_fmaf(g[q], f[q], dot);
                        o[q] = on ? w * g[q] : 0.f;
                    }
                    st_chunk(dy + j, repack<T>(o));
                } else {
                    for (uint32_t q = j; q < a.width; ++q) {
                        const float gq = on ? widen(T{}, d[q]) : 0.f;
                        if (on) dot = __builtin_fmaf(gq, widen(T{}, y[q]), dot);
                        dy[q] = narrow(T{}, on ? w * gq : 0.f);
                    }
                }
            }
        }
        dot = wave_sum(dot);
        if (lane == 0) a.dweights_w[r] = on ? dot : 0.f;
    }
}

uint32_t cap(int64_t n) { return (uint32_t)(n < 1 ? 1 : n < (1 << 20) ? n : (1 << 20)); }

}  // namespace

hipError_t launch_sort_plan(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_SORT_PLAN;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel((const void*)&sort_plan, dim3(a.n_experts + 1), dim3(PThreads), args, 0, s);
}

hipError_t launch_sort_gather(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_SORT_GATHER;
    const void* fn = a.dtype == 0 ? (const void*)&sort_gather<uint32_t> : (const void*)&sort_gather<uint16_t>;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, dim3(cap((int64_t)a.m * a.top_k)), dim3(CThreads), args, 0, s);
}

hipError_t launch_combine(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_COMBINE;
    const bool w = a.weights != nullptr;
    const void* fn = a.dtype == 0   ? (w ? (const void*)&combine<TF32, true> : (const void*)&combine<TF32, false>)
                     : a.dtype == 1 ? (w ? (const void*)&combine<TF16, true> : (const void*)&combine<TF16, false>)
                                    : (w ? (const void*)&combine<TBF16, true> : (const void*)&combine<TBF16, false>);
    const int64_t per = CThreads * (a.dtype == 0 ? 4 : 8);
    const int64_t pieces = (a.width + per - 1) / per;  // width < 2^26: at most 2^16
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, dim3(cap(a.m < 65536 ? a.m : 65536), (uint32_t)pieces), dim3(CThreads), args, 0, s);
}

hipError_t launch_combine_grad(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_COMBINE_GRAD;
    const void* fn = a.dtype == 0   ? (const void*)&combine_grad<TF32>
                     : a.dtype == 1 ? (const void*)&combine_grad<TF16>
                                    : (const void*)&combine_grad<TBF16>;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, dim3(cap(((int64_t)a.m * a.top_k + CWaves - 1) / CWaves)), dim3(CThreads), args, 0, s);
}

}  // namespace mmk
