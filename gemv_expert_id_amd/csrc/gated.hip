// Gated feed-forward block: h = act(x G^T) * (x U^T), and the gradients of its
// pre-activations (mm.h, "Feed-forward block").
#include "ffn_strided.hpp"

namespace mmk {

namespace {

// dpre from saved pre-activations, element by element: 16 bytes of the gate's
// half, of the up projection's and of dh in, 16 bytes of each half out. Bound by
// memory: 4096 x 22016 bf16 in 90 us, 5.0 TB/s. A block takes 2^sh chunks of a row by 256 / 2^sh rows. In place (pre ==
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

// Few rows by few columns over a long contraction (dpre . w of a small batch): 16 FM
// rows x 16 columns a block, whose 16 waves take every 16th step of 32 of the
// contraction, read both operands straight into fragments, DEP steps in flight, and are
// summed in order through LDS. A wave's lanes hold 8 rows of w at a column each, so w's
// loads are single elements: 16 neighbours a row. Bound by the CU's own load path, for
// few blocks share one contraction: 3.5 times what the bytes of w take, as are the forms
// beside it. us, here and in the form that would be taken else: f32 8 x 49 over 21376 53.7
// and 88.6, 16 x 1024 over 8198 29.0 and 36.4, 32 x 64 over 2000 8.8 and 9.7, 32 x 130 over
// 600 7.8 and 4.7; bf16 8 x 49 over 21376 33.9 and 86.9, 16 x 4096 over 22016 119 and 122,
// 32 x 1024 over 8198 28.4 and 33.8, 32 x 256 over 4096 12.4 and 13.9, 16 x 1601 over 700
// 5.3 and 4.8. Taken although slower: 16 x 4096 over 8192 f16 40.3 and 32.0, over 4096
// bf16 20.4 and 16.5.
template <class T, int FM>
__global__ __launch_bounds__(1024) void long_product(FfnArgs a) {
    using S = typename T::store_t;
    using M = MmaOf<T>;
    constexpr int P = kParts<T>, DEP = T::code == 0 && FM > 1 ? 2 : 4;
    __shared__ f32x4 part[16][FM][64];
    const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16, ldw = a.ldw / (int64_t)sizeof(S);
    const auto w_col = [&](int c, int) {  // columns past the end repeat the last
        return static_cast<const S*>(a.w) + (n0 + c < a.n ? n0 + c : a.n - 1);
    };
    const S* w = w_col(lr, 0);
    const auto x_row = [&](int row, int i) {
        return static_cast<const S*>(a.x) + (i * 16 + row < a.m ? i * 16 + row : a.m - 1) * (a.ldx / (int64_t)sizeof(S));
    };
    const S* x[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) x[i] = x_row(lr, i);
    f32x4 acc[FM][1], low[FM][1];
    uint32_t lost = 0;  // (parts_of)
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[i][0] = low[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    const auto multiply = [&](const S (&ew)[8], const Pack<S, 8> (&ex)[FM]) {
        uint32_t pw[P][4], px[P][4];
        parts_of<T, 8>(ew, pw, lost);
        u32x4 fw[P], fx[P];
#pragma unroll
        for (int q = 0; q < P; ++q) fw[q] = u32x4{pw[q][0], pw[q][1], pw[q][2], pw[q][3]};
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            parts_of<T, 8>(ex[i].v, px, lost);
#pragma unroll
            for (int q = 0; q < P; ++q) fx[q] = u32x4{px[q][0], px[q][1], px[q][2], px[q][3]};
            if constexpr (P == 3) {
                low[i][0] = step_mma<M>(fw[2], fx[0], low[i][0]);
                low[i][0] = step_mma<M>(fw[0], fx[2], low[i][0]);
                low[i][0] = step_mma<M>(fw[1], fx[1], low[i][0]);
                low[i][0] = step_mma<M>(fw[1], fx[0], low[i][0]);
                low[i][0] = step_mma<M>(fw[0], fx[1], low[i][0]);
            }
            acc[i][0] = step_mma<M>(fw[0], fx[0], acc[i][0]);
        }
    };
    const int64_t whole = a.k / 32;  // steps
    int64_t s = wave;
    for (; s + 16 * (DEP - 1) < whole; s += 16 * DEP) {
        S ew[DEP][8];
        Pack<S, 8> ex[DEP][FM];
#pragma unroll
        for (int d = 0; d < DEP; ++d) {
            const int64_t r = (s + 16 * d) * 32 + 8 * lq;
#pragma unroll
            for (int i = 0; i < FM; ++i) ex[d][i] = *reinterpret_cast<const Pack<S, 8>*>(x[i] + r);
#pragma unroll
            for (int e = 0; e < 8; ++e) ew[d][e] = w[(r + e) * ldw];
        }
#pragma unroll
        for (int d = 0; d < DEP; ++d) multiply(ew[d], ex[d]);
    }
    for (; s * 32 < a.k; s += 16) {  // the rest; rows past the end are zeros in both
        const int64_t r = s * 32 + 8 * lq;
        S ew[8];
        Pack<S, 8> ex[FM];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool in = r + e < a.k;
            ew[e] = in ? w[(r + e) * ldw] : S(0);
#pragma unroll
            for (int i = 0; i < FM; ++i) ex[i].v[e] = in ? x[i][r + e] : S(0);
        }
        multiply(ew, ex);
    }
    if constexpr (P == 3) {
        f32_join<16, true, false>(a.k, wave, parts_lost(lost), x_row, 1, w_col, ldw, acc, low);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) part[wave][i][lane] = acc[i][0];
    __syncthreads();
    if (wave >= FM) return;
    f32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int g = 1; g < 16; ++g) sum += part[g][wave][lane];
    const PlainOut<T> out{a};
    if (wave * 16 + lr < a.m) out.one(wave * 16 + lr, n0 + 4 * lq, sum);
}
template <class T>
hipError_t long_product(const FfnArgs& o, hipStream_t s) {
    const dim3 grid((unsigned)((o.n + 15) / 16));
    void* args[] = {const_cast<FfnArgs*>(&o)};
    const void* fn = o.m <= 16 ? (const void*)&long_product<T, 1> : (const void*)&long_product<T, 2>;
    return hipLaunchKernel(fn, grid, dim3(1024), args, 0, s);
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
// more of them than CUs, by two beyond; 256 x 128 tiles where they make one round that
// fills more than half of the CUs (`one_round`) or many, over a long contraction (us,
// f16: 1024 x 4096 over 4096, 256 tiles of 128 x 128, 35.8, 45.5 and 51.0; 2816 x 2048 over 3001
// transposed, 352, 56.8, 50.1 and 45.4; 11008 x 2048 over 512, 1376, 52.3, 40.7 and 45.2;
// over 4096, 225, 201 and 188).
template <class T>
hipError_t chunked_product(const GemmArgs& g, const FfnArgs& o, int64_t tiles, bool one_round, hipStream_t s) {
    if (tiles <= 256) return pipe_product<T, PipeShape<2, 4, 4, 2, 4>>(g, o, s);
    if (one_round || (tiles > 1024 && g.k >= 2048)) return pipe_product<T, PipeShape<4, 2, 4, 4, 3>>(g, o, s);
    return pipe_product<T, PipeShape<2, 4, 4, 2, 2>>(g, o, s);
}

}  // namespace

// dpre . w (both as stored: NN) or dpre^T . x (TN), of dpre as it was rounded: it is an
// output that a caller keeps, and in 16 bits one matrix instruction takes it where two
// parts would need two. That adds to the error: 0.0023 of the norm in bf16, where unrounded
// dpre gives 0.0017 (the rounding of dx and dw themselves); 0.00029 and 0.00021 in f16.
//
// Products whose contraction the pipelined GEMM takes whole go to it, and large TN ones of
// any contraction (it reads zeros past the end), unless the tiles here leave fewer CUs idle
// in their last round; others take the forms here: pipelined ones where rows hold whole
// 16-byte pieces and 128 x 128 tiles are more than 64, tiles of any alignment else. us,
// f16, GEMM and here: 4096 x 4096 over 4096, 111 and 129; 3001 x 2048 over 2816, 48.6 and
// 42.2, over 11008, 177 and 136; 11008 x 2048 over 1024 transposed, 344 tiles of 256 x 256,
// 75.5 and 66.5, 22016 x 4096 over 4096, 1376 tiles, 710 and 810; 512 x 2048 over 2816, 64
// tiles, any alignment 20.1, pipelined 22.4, GEMM 20.5.
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
    // Rounds of 256 x 256 tiles (one costs 1.7 to 1.9 of the other) and of 256 x 128 tiles.
    const int64_t tall = (g.m + 255) / 256, squares = tall * ((g.n + 255) / 256), halves = tall * ((g.n + 127) / 128);
    const bool one_round = halves > 128 && halves <= 256 && g.k >= 1024;
    const bool fuller = (squares > 128 && 10 * ((halves + 255) / 256) < 17 * ((squares + 255) / 256)) ||
                        (one_round && !g.ta && g.k >= 2048);
    if (gemm && tiles > 64 && !fuller && (whole || (g.ta && squares >= 192))) {
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
    if (!g.ta && g.m <= 32 && g.n <= 4096 && g.k >= (g.dtype == 0 || g.m <= 16 ? 1024 : 8192))
        return g.dtype == 0   ? long_product<TF32>(o, s)
               : g.dtype == 1 ? long_product<TF16>(o, s)
                              : long_product<TBF16>(o, s);
    if (chunked && tiles > 64)
        return g.dtype == 1 ? chunked_product<TF16>(g, o, tiles, one_round, s)
                            : chunked_product<TBF16>(g, o, tiles, one_round, s);
    if (g.dtype == 0) return g.ta ? run_f32_product<true>(o, s) : run_f32_product<false>(o, s);
    return g.dtype == 1 ? tile_product<TF16>(g, o, s) : tile_product<TBF16>(g, o, s);
}

hipError_t launch_gated(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_GATED;
    return a.dtype == 0   ? run_ffn_f32<GatedOut<TF32>>(a, s, L)
           : a.dtype == 1 ? run_ffn<GatedOut<TF16>>(a, s, L)
                          : run_ffn<GatedOut<TBF16>>(a, s, L);
}

hipError_t launch_gated_again(const FfnArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_GATED_GRAD;
    return a.dtype == 0   ? run_ffn_f32<GradOut<TF32>>(a, s, L)
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
