// Gated feed-forward block: h = act(x G^T) * (x U^T), and the gradients of its
// pre-activations (mm.h, "Feed-forward block").
#include "ffn_pipe.hpp"

namespace mmk {

namespace {

// dpre from saved pre-activations, element by element: 16 bytes of the gate's
// half, of the up projection's and of dh in, 16 bytes of each half out. Bound by
// memory. A block takes 2^sh chunks of a row by 256 / 2^sh rows. In place (pre ==
// dpre) every element is read before the same lane writes it.
template <class T>
__global__ __launch_bounds__(256) void gated_grad(FfnArgs a, int sh) {
    using S = typename T::store_t;
    constexpr int V = T::Elems16;
    using U16 = Pack<S, V>;
    const int64_t c = (int64_t)blockIdx.x * (1 << sh) + (threadIdx.x & ((1 << sh) - 1));
    const int64_t col = c * V;
    if (col >= a.n) return;
    const int valid = (int)(a.n - col < V ? a.n - col : V);
    const int64_t rows = 256 >> sh;
    for (int64_t r = blockIdx.y * rows + (threadIdx.x >> sh); r < a.m; r += gridDim.y * rows) {
        const S* g = static_cast<const S*>(a.pre) + r * a.ldpre + col;
        const S* u = g + a.n;
        const S* d = static_cast<const S*>(a.dh) + r * a.ldy + col;
        S* dg = static_cast<S*>(a.pre_w) + r * a.ldpre + col;
        S* du = dg + a.n;
        S gs[V], us[V], ds[V];
        if (valid == V) {
            *reinterpret_cast<U16*>(gs) = *reinterpret_cast<const U16*>(g);
            *reinterpret_cast<U16*>(us) = *reinterpret_cast<const U16*>(u);
            *reinterpret_cast<U16*>(ds) = *reinterpret_cast<const U16*>(d);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                gs[i] = i < valid ? g[i] : S(0);
                us[i] = i < valid ? u[i] : S(0);
                ds[i] = i < valid ? d[i] : S(0);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float x, y;
            gate_grad(a.gate, widen(T{}, gs[i]), widen(T{}, us[i]), widen(T{}, ds[i]), &x, &y);
            gs[i] = narrow(T{}, x);
            us[i] = narrow(T{}, y);
        }
        if (valid == V) {
            *reinterpret_cast<U16*>(dg) = *reinterpret_cast<const U16*>(gs);
            *reinterpret_cast<U16*>(du) = *reinterpret_cast<const U16*>(us);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < valid) {
                    dg[i] = gs[i];
                    du[i] = us[i];
                }
        }
    }
}

template <class T>
hipError_t tile_product(const GemmArgs& g, const FfnArgs& o, hipStream_t s) {
    const TileArgs t{g.A, g.B, g.m, g.n, g.k, g.lda, g.ldb, 0};
    return g.ta ? run_ffn_tile<PlainOut<T>, false, false>(t, o, s) : run_ffn_tile<PlainOut<T>, true, false>(t, o, s);
}
template <class T, class Z>
hipError_t pipe_product(const GemmArgs& g, const FfnArgs& o, hipStream_t s) {
    return g.ta ? run_ffn_pipe<PlainOut<T>, Z, false, false>(o, s) : run_ffn_pipe<PlainOut<T>, Z, true, false>(o, s);
}
// 16-byte pieces in both operands: 128 x 128 tiles by one block a CU while there are no
// more of them than CUs, by two up to 1024, 256 x 128 tiles beyond (us, bf16: 1024 x
// 4096 over 8192, 256 tiles, 73.7 and 111; 3001 x 2048 over 2816, 46.3, 42.0 and 42.1;
// 8192 x 8192 over 8192, 1101, 1031 and 910).
template <class T>
hipError_t chunked_product(const GemmArgs& g, const FfnArgs& o, int64_t tiles, hipStream_t s) {
    if (tiles <= 256) return pipe_product<T, PipeShape<2, 4, 4, 2, 4>>(g, o, s);
    if (tiles <= 1024) return pipe_product<T, PipeShape<2, 4, 4, 2, 2>>(g, o, s);
    return pipe_product<T, PipeShape<4, 2, 4, 4, 3>>(g, o, s);
}

}  // namespace

// dpre . w (both as stored: NN) or dpre^T . x (TN). Products whose contraction the
// pipelined GEMM takes whole go to it, and large TN ones of any contraction (it reads
// zeros past the end); others take the forms here: pipelined ones where rows hold
// whole 16-byte pieces and 128 x 128 tiles are more than 64, tiles of any alignment
// else (us, bf16: 512 x 2048 over 2816, 64 tiles, 20.1 in those against 22.4 pipelined
// and 20.5 by the GEMM; 2816 x 2048 over 3001, 352 tiles, 89 against 46).
hipError_t launch_gated_product(const GemmArgs& g, hipStream_t s, Launched* L) {
    const auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const int64_t es = g.dtype == 0 ? 4 : 2;
    const int64_t span_a = g.ta ? (g.k + 127) * g.lda + g.m : (g.m - 1) * g.lda + g.k;
    const int64_t span_b = (g.k + 127) * g.ldb + g.n;
    const int64_t tiles = ((g.m + 127) / 128) * ((g.n + 127) / 128);
    const bool chunked = g.dtype != 0 && al16(g.A) && al16(g.B) && g.lda % 8 == 0 && g.ldb % 8 == 0 &&
                         g.lda < (1 << 21) && g.ldb < (1 << 21) && (g.ta || g.k % 8 == 0);
    const bool gemm = chunked && (reinterpret_cast<uintptr_t>(g.C) & 7) == 0 && g.ldc % 4 == 0 &&
                      span_a < (1ll << 30) && span_b < (1ll << 30);
    const bool whole = g.k % 128 == 0 && g.k >= 256;
    if (gemm && tiles > 64 && (whole || (g.ta && ((g.m + 255) / 256) * ((g.n + 255) / 256) >= 192))) {
        GemmArgs q = g;
        q.ragged_k = 1;
        return launch_gemm(q, s, L);
    }
    L->kernel = MM_KERNEL_GATED_GRAD;
    FfnArgs o{};
    o.x = g.A;
    o.w = g.B;
    o.y = g.C;
    o.m = g.m;
    o.n = g.n;
    o.k = g.k;
    o.ldx = g.lda * es;
    o.ldw = g.ldb * es;
    o.ldy = g.ldc;
    if (chunked && tiles > 64)
        return g.dtype == 1 ? chunked_product<TF16>(g, o, tiles, s) : chunked_product<TBF16>(g, o, tiles, s);
    return g.dtype == 0   ? tile_product<TF32>(g, o, s)
           : g.dtype == 1 ? tile_product<TF16>(g, o, s)
                          : tile_product<TBF16>(g, o, s);
}

hipError_t launch_gated(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_GATED;
    return a.dtype == 0   ? run_ffn<GatedOut<TF32>>(a, s, L)
           : a.dtype == 1 ? run_ffn<GatedOut<TF16>>(a, s, L)
                          : run_ffn<GatedOut<TBF16>>(a, s, L);
}

hipError_t launch_gated_again(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_GATED_GRAD;
    return a.dtype == 0   ? run_ffn<GradOut<TF32>>(a, s, L)
           : a.dtype == 1 ? run_ffn<GradOut<TF16>>(a, s, L)
                          : run_ffn<GradOut<TBF16>>(a, s, L);
}

hipError_t launch_gated_grad(const FfnArgs& a, hipStream_t s, Launched* L) {
    const int v = a.dtype == 0 ? 4 : 8;
    const int64_t chunks = (a.n + v - 1) / v;
    int sh = 0;
    while (sh < 8 && (1 << sh) < chunks) ++sh;
    const int64_t rows = 256 >> sh, gx = (chunks + (1 << sh) - 1) >> sh;
    const int64_t gy = (a.m + rows - 1) / rows;
    const dim3 grid((unsigned)gx, (unsigned)(gy < 65535 ? gy : 65535));
    const void* fn = a.dtype == 0   ? (const void*)&gated_grad<TF32>
                     : a.dtype == 1 ? (const void*)&gated_grad<TF16>
                                    : (const void*)&gated_grad<TBF16>;
    void* args[] = {const_cast<FfnArgs*>(&a), &sh};
    L->kernel = MM_KERNEL_GATED_GRAD;
    return hipLaunchKernel(fn, grid, dim3(256), args, 0, s);
}

}  // namespace mmk
