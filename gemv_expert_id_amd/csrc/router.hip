// Router of a mixture-of-experts layer and its gradient.
//
// topk: one wave per token. Lane l holds the logits of experts l*EPL ..
// l*EPL + EPL - 1, so the lowest expert of equal logits is the lowest index of
// the lowest lane. A logit is compared as an unsigned key in the order of the
// floats (0 for what may not be chosen: -inf, NaN, past the row's end). Each
// of the top_k rounds takes the wave's largest key, finds its first lane with
// a ballot, and clears that one key; lane s keeps the s-th choice.
//
// topk_grad: one wave per token; the gradients of the chosen experts are
// scattered through LDS, and the softmax is taken again from the logits.
#include "common.hpp"
#include "kernels.hpp"

namespace mmk {

namespace {

constexpr int RThreads = 256;
constexpr int RWaves = RThreads / kWave;
constexpr uint32_t kNone = 0xFFFFFFFFu;

// Unsigned order of the floats; 0 below every logit that can be chosen.
__device__ __forceinline__ uint32_t sort_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);  // -0 and +0 are equal logits
    const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return v > -INFINITY ? k : 0u;  // false for NaN too
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t w = (uint32_t)__shfl_xor((int)v, o, kWave);
        v = v > w ? v : w;
    }
    return v;
}

template <class T, int EPL>
__global__ __launch_bounds__(RThreads) void topk(TopkArgs a) {
    using S = typename T::store_t;
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t E = a.n_experts;
    for (int64_t t = (int64_t)blockIdx.x * RWaves + threadIdx.x / kWave; t < a.m;
         t += (int64_t)gridDim.x * RWaves) {
        const S* row = static_cast<const S*>(a.logits) + t * a.ld;
        uint32_t key[EPL];
        float val[EPL];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t e = lane * EPL + j;
            val[j] = e < E ? widen(T{}, row[e]) : -INFINITY;
            key[j] = sort_key(val[j]);
            nan |= val[j] != val[j];
        }
        const bool any_nan = __ballot(nan) != 0;
        uint32_t top_key = 0, id = kNone, top0 = 0;
        for (uint32_t s = 0; s < a.top_k; ++s) {
            uint32_t best = key[0];
#pragma unroll
            for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
            const uint32_t m = wave_max_u32(best);
            if (m == 0) break;
            if (s == 0) top0 = m;
            const int first = __ffsll((unsigned long long)__ballot(best == m)) - 1;
            int at = EPL - 1;
#pragma unroll
            for (int j = EPL - 2; j >= 0; --j) at = key[j] == m ? j : at;
            if (lane == first) {
#pragma unroll
                for (int j = 0; j < EPL; ++j) key[j] = j == at ? 0u : key[j];
            }
            const uint32_t e = (uint32_t)__shfl(lane * EPL + at, first, kWave);
            if (lane == (int)s) { top_key = m; id = e; }
        }
        // exp(l - largest): the chosen by their keys, all of them by their values.
        const float peak = key_value(top0);
        const float mine = id != kNone ? expf(key_value(top_key) - peak) : 0.f;
        float total = mine;
        if (!a.renormalize) {
            total = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) total += top0 && val[j] != -INFINITY ? expf(val[j] - peak) : 0.f;
        }
        total = wave_sum(total);
        if (lane < (int)a.top_k) {
            const int64_t o = t * a.top_k + lane;
            a.ids_w[o] = id;
            a.weights_w[o] = id == kNone ? 0.f : any_nan ? __uint_as_float(0x7FC00000u) : mine / total;
        }
    }
}

template <class T, int EPL>
__global__ __launch_bounds__(RThreads) void topk_grad(TopkArgs a) {
    using S = typename T::store_t;
    __shared__ float g_all[RWaves][EPL * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    float* gs = g_all[threadIdx.x / kWave];
    const uint32_t E = a.n_experts;
    const int64_t rounds = (a.m + (int64_t)gridDim.x * RWaves - 1) / ((int64_t)gridDim.x * RWaves);
    for (int64_t q = 0; q < rounds; ++q) {
        const int64_t t = (q * gridDim.x + blockIdx.x) * RWaves + threadIdx.x / kWave;
        const bool live = t < a.m;
        const S* row = static_cast<const S*>(a.logits) + (live ? t : 0) * a.ld;
        uint32_t id = kNone;
        float g = 0.f;
        if (live && lane < (int)a.top_k) {
            id = a.ids[t * a.top_k + lane];
            if (id < E) g = a.dweights[t * a.top_k + lane];
        }
        const bool has = id < E;
        float val[EPL], p[EPL];
        float peak = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t e = lane + j * kWave;
            val[j] = e < E ? widen(T{}, row[e]) : -INFINITY;
            gs[e] = 0.f;
        }
        __syncthreads();
        float mine = -INFINITY;
        if (has) {
            gs[id] = 1.f;
            mine = widen(T{}, row[id]);
        }
        __syncthreads();
        // Softmax over all experts, or over the chosen (marked in LDS).
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (a.renormalize && gs[lane + j * kWave] == 0.f) val[j] = -INFINITY;
            peak = fmaxf(peak, val[j]);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor(peak, o, kWave));
        float total = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            p[j] = val[j] == -INFINITY ? 0.f : expf(val[j] - peak);
            total += p[j];
        }
        total = wave_sum(total);
        const float inv = 1.f / total;
        const float dot = wave_sum(has ? g * (expf(mine - peak) * inv) : 0.f);
        __syncthreads();
        if (has) gs[id] = g;
        __syncthreads();
        const bool any = __ballot(has) != 0;
        if (live) {
            S* out = static_cast<S*>(a.dlogits) + t * a.ld;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const uint32_t e = lane + j * kWave;
                const float d = !any || val[j] == -INFINITY ? 0.f : p[j] * inv * (gs[e] - dot);
                if (e < E) out[e] = narrow(T{}, d);
            }
        }
        __syncthreads();
    }
}

template <class T>
const void* pick(bool grad, uint32_t E) {
    const int epl = (int)((E + kWave - 1) / kWave);
#define MM_EPL(n) \
    if (epl <= n) return grad ? (const void*)&topk_grad<T, n> : (const void*)&topk<T, n>;
    MM_EPL(1) MM_EPL(2) MM_EPL(4) MM_EPL(8) MM_EPL(16)
#undef MM_EPL
    return nullptr;
}

}  // namespace

hipError_t launch_topk(const TopkArgs& a, bool grad, hipStream_t s, Launched* L) {
    L->kernel = grad ? MM_KERNEL_TOPK_GRAD : MM_KERNEL_TOPK;
    const void* fn = a.dtype == 0   ? pick<TF32>(grad, a.n_experts)
                     : a.dtype == 1 ? pick<TF16>(grad, a.n_experts)
                                    : pick<TBF16>(grad, a.n_experts);
    if (!fn) return hipErrorInvalidValue;
    const int64_t blocks = (a.m + RWaves - 1) / RWaves;
    void* args[] = {const_cast<TopkArgs*>(&a)};
    return hipLaunchKernel(fn, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(RThreads),
                           args, 0, s);
}

}  // namespace mmk
