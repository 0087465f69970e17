// Router of a mixture-of-experts layer and its gradient.
//
// A logit is compared as an unsigned key in the order of the floats (0 for
// what may not be chosen: -inf, NaN, past the row's end); lanes hold
// neighbouring experts, so the lowest of equal logits is the lowest index of
// the lowest lane. Reductions are DPP row operations: an LDS shuffle costs
// about 100 clocks of latency in each of a reduction's steps, a DPP step about 8.
//
// topk_rows (16-bit logits, up to 512 experts, 16 slots): 16 lanes a token,
// four tokens a wave. The key is 16 bits, so a register holds it above the
// expert's complement and every key is unique. Each lane sorts its own
// keys with an odd-even merge network; a round takes the largest head of the
// 16 lanes and the lane that owns it moves its list up. Bound by vector issue:
// 16384 x 256 bf16, top 8, in 6.5 us (560 instructions for four tokens; one wave a
// token 16.1 us; the logits alone would take 1.8 us).
//
// topk (the rest): one wave a token; a round takes the wave's largest key,
// finds its first lane with a ballot, and clears that one key. One token of 64
// f32 experts: 2.4 us, a launch and one memory round trip.
//
// topk_grad: one wave a token; the chosen experts are marked in LDS that the wave
// alone uses, and the softmax is taken again. 8191 x 97 f32 in 4.6 us, 1.5 TB/s:
// two memory round trips (ids and logits, then the stores).
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

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {  // lanes without a source get 0
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
// A reduction over the wave with identity 0: lane 63 ends with the whole, read by all.
template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
    v = f(v, dpp<0x111>(v));       // row_shr:1
    v = f(v, dpp<0x112>(v));       // row_shr:2
    v = f(v, dpp<0x114>(v));       // row_shr:4
    v = f(v, dpp<0x118>(v));       // row_shr:8
    v = f(v, dpp<0x142, 0xA>(v));  // row_bcast:15
    v = f(v, dpp<0x143, 0xC>(v));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
// The same over each row of 16 lanes, the whole in every lane.
template <class F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f) {
    v = f(v, dpp<0x128>(v));  // row_ror:8
    v = f(v, dpp<0x124>(v));
    v = f(v, dpp<0x122>(v));
    v = f(v, dpp<0x121>(v));
    return v;
}
struct MaxU {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct AddF {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }
};
__device__ __forceinline__ float wave_add(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), AddF{}));
}

// Sorts N (a power of two) keys, largest first: Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t x = k[i + j], y = k[i + j + q];
                        k[i + j] = x > y ? x : y;
                        k[i + j + q] = x > y ? y : x;
                    }
}

// The order of a 16-bit logit as a number around 0x8000 (both zeros give
// 0x8000), and back. kInf: the magnitude of infinity; above it lie the NaNs.
template <class T>
constexpr uint32_t kInf = T::code == 1 ? 0x7C00u : 0x7F80u;
__device__ __forceinline__ uint32_t order16(uint32_t bits) {
    const uint32_t mag = bits & 0x7FFFu;
    return bits & 0x8000u ? 0x8000u - mag : 0x8000u + mag;
}
template <class T>
__device__ __forceinline__ float value16(uint32_t order) {
    return widen(T{}, (uint16_t)(order < 0x8000u ? 0x8000u | (0x8000u - order) : order - 0x8000u));
}

// 16-bit logits, E <= 16 * EPL <= 512, top_k <= KEEP or, where KEEP is EPL, 16. A
// lane's list can lose no more than KEEP keys, so the others need not move up.
template <class T, int EPL, int KEEP>
__global__ __launch_bounds__(RThreads) void topk_rows(TopkArgs a) {
    constexpr int TPB = RThreads / 16;  // tokens of a block
    const int l = threadIdx.x & 15;
    const uint32_t E = a.n_experts;
    for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.m; t0 += (int64_t)gridDim.x * TPB) {
        const int64_t t = t0 + threadIdx.x / 16;
        const bool live = t < a.m;
        const uint16_t* row = static_cast<const uint16_t*>(a.logits) + (live ? t : 0) * a.ld;
        uint32_t key[EPL];
        const uint32_t e0 = l * EPL;
        struct __attribute__((packed, aligned(2))) Pack { uint16_t h[EPL]; };
        Pack raw;
        if (e0 + EPL <= E) {
            raw = *reinterpret_cast<const Pack*>(row + e0);
        } else {  // -inf past the row's end: never chosen
#pragma unroll
            for (int j = 0; j < EPL; ++j) raw.h[j] = e0 + j < E ? row[e0 + j] : (uint16_t)(0x8000u | kInf<T>);
        }
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t o = order16(raw.h[j]);
            // What can be chosen lies above -inf and up to +inf.
            key[j] = o - (0x8001u - kInf<T>) < 2 * kInf<T> ? o << 16 | (0xFFFFu - j - e0) : 0u;
            nan |= (raw.h[j] & 0x7FFFu) > kInf<T>;
        }
        const uint64_t nans = __ballot(nan);
        const bool any_nan = (nans >> (threadIdx.x & 48) & 0xFFFFu) != 0;
        sort_keys<EPL>(key);
        const auto value = [](uint32_t k) { return value16<T>(k >> 16); };
        const uint32_t first = row_reduce(key[0], MaxU{});
        const float peak = value(first);
        float total = 0.f;
        if (!a.renormalize) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) total += key[j] ? expf(value(key[j]) - peak) : 0.f;
        }
        uint32_t mine = 0;
        for (int s = 0; s < (int)a.top_k; ++s) {
            const uint32_t m = s == 0 ? first : row_reduce(key[0], MaxU{});
            mine = l == s ? m : mine;
            const bool own = key[0] == m;
#pragma unroll
            for (int j = 0; j < KEEP - 1; ++j) key[j] = own ? key[j + 1] : key[j];
            key[KEEP - 1] = own ? 0u : key[KEEP - 1];
        }
        const float w = mine ? expf(value(mine) - peak) : 0.f;
        if (a.renormalize) total = w;
        total = __uint_as_float(row_reduce(__float_as_uint(total), AddF{}));
        if (live && l < (int)a.top_k) {
            const int64_t o = t * a.top_k + l;
            a.ids_w[o] = mine ? 0xFFFFu - (mine & 0xFFFFu) : kNone;
            a.weights_w[o] = !mine ? 0.f : any_nan ? __uint_as_float(0x7FC00000u) : w / total;
        }
    }
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
            const uint32_t m = wave_reduce(best, MaxU{});
            if (m == 0) break;
            if (s == 0) top0 = m;
            const int first = __ffsll((unsigned long long)__ballot(best == m)) - 1;
            int at = EPL - 1;
#pragma unroll
            for (int j = EPL - 2; j >= 0; --j) at = key[j] == m ? j : at;
#pragma unroll
            for (int j = 0; j < EPL; ++j) key[j] = lane == first && j == at ? 0u : key[j];
            const uint32_t e = (uint32_t)__builtin_amdgcn_readlane(lane * EPL + at, first);
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
        total = wave_add(total);
        if (lane < (int)a.top_k) {
            const int64_t o = t * a.top_k + lane;
            a.ids_w[o] = id;
            a.weights_w[o] = id == kNone ? 0.f : any_nan ? __uint_as_float(0x7FC00000u) : mine / total;
        }
    }
}

// Orders a wave's own LDS accesses: they execute in order, the compiler needs telling.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <class T, int EPL>
__global__ __launch_bounds__(RThreads) void topk_grad(TopkArgs a) {
    using S = typename T::store_t;
    __shared__ uint32_t slot_all[RWaves][EPL * kWave];
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t* slot = slot_all[threadIdx.x / kWave];  // 1 + the slot that chose an expert, or 0
    const uint32_t E = a.n_experts;
    for (int64_t t = (int64_t)blockIdx.x * RWaves + threadIdx.x / kWave; t < a.m;
         t += (int64_t)gridDim.x * RWaves) {
        const S* row = static_cast<const S*>(a.logits) + t * a.ld;
        uint32_t id = kNone;
        float g = 0.f;
        if (lane < (int)a.top_k) {
            id = a.ids[t * a.top_k + lane];
            g = a.dweights[t * a.top_k + lane];
        }
        float val[EPL];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t e = lane + j * kWave;
            val[j] = e < E ? widen(T{}, row[e]) : -INFINITY;
            nan |= val[j] != val[j];
            slot[e] = 0;
        }
        // A NaN makes the token's weights NaN whether it was chosen or not.
        const bool any_nan = __ballot(nan) != 0;
        wave_lds_fence();
        if (id < E) slot[id] = lane + 1;
        wave_lds_fence();
        const bool any = __ballot(id < E) != 0;
        float ge[EPL], p[EPL];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t s = slot[lane + j * kWave];
            const float gs = __shfl(g, (int)s - 1, kWave);
            ge[j] = s ? gs : 0.f;
            if (a.renormalize && !s) val[j] = -INFINITY;
            const uint32_t k = sort_key(val[j]);
            top = k > top ? k : top;
        }
        const float peak = key_value(wave_reduce(top, MaxU{}));
        float total = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            p[j] = val[j] == -INFINITY ? 0.f : expf(val[j] - peak);
            total += p[j];
            dot += ge[j] * p[j];
        }
        const float inv = any_nan ? __uint_as_float(0x7FC00000u) : 1.f / wave_add(total);
        dot = wave_add(dot) * inv;
        S* out = static_cast<S*>(a.dlogits) + t * a.ld;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const uint32_t e = lane + j * kWave;
            const float d = !any || val[j] == -INFINITY ? 0.f : p[j] * inv * (ge[j] - dot);
            if (e < E) out[e] = narrow(T{}, d);
        }
        wave_lds_fence();
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
template <class T>
const void* pick_rows(uint32_t E, uint32_t top_k) {
    const int epl = (int)((E + 15) / 16);
#define MM_EPL(n) \
    if (epl <= n) return top_k <= 8 ? (const void*)&topk_rows<T, n, (n < 8 ? n : 8)> : (const void*)&topk_rows<T, n, n>;
    MM_EPL(1) MM_EPL(2) MM_EPL(4) MM_EPL(8) MM_EPL(16) MM_EPL(32)
#undef MM_EPL
    return nullptr;
}

}  // namespace

hipError_t launch_topk(const TopkArgs& a, bool grad, hipStream_t s, Launched* L) {
    L->kernel = grad ? MM_KERNEL_TOPK_GRAD : MM_KERNEL_TOPK;
    const bool rows = !grad && a.dtype != 0 && a.n_experts <= 512 && a.top_k <= 16;
    L->variant = rows ? 16 : kWave;
    const void* fn = rows            ? (a.dtype == 1 ? pick_rows<TF16>(a.n_experts, a.top_k) : pick_rows<TBF16>(a.n_experts, a.top_k))
                     : a.dtype == 0   ? pick<TF32>(grad, a.n_experts)
                     : a.dtype == 1 ? pick<TF16>(grad, a.n_experts)
                                    : pick<TBF16>(grad, a.n_experts);
    if (!fn) return hipErrorInvalidValue;
    const int64_t per = rows ? RThreads / 16 : RWaves;
    const int64_t blocks = (a.m + per - 1) / per;
    void* args[] = {const_cast<TopkArgs*>(&a)};
    return hipLaunchKernel(fn, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(RThreads),
                           args, 0, s);
}

}  // namespace mmk
