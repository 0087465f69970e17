// Products with 4-bit weights and group scales, y = sum over groups of
// s * (q . x) + b * sum(x), on matrix instructions.
//
// A wave takes 16 rows of W and a contiguous piece of k, 128 elements (64
// bytes of codes a row) at a step: lane l loads the 16 bytes at chunk l / 16 of
// row l % 16. Four such waves of a block take the pieces of k and join their
// sums through LDS. The codes are the B operand of v_mfma_f32_16x16x32 (column
// = row of W), the activations the A operand (row = token):
//   - A code becomes an operand by placing its four bits in the mantissa of
//     16.0, which is 16 + q, exact in f16 and bf16: one shift and one
//     and-or for two codes, no conversion. The 16 is taken back with the
//     group's sum of x, which the same instruction gives from a constant
//     operand: D0 = (-16) . x, so q . x = (16 + q) . x + D0 and
//     b * sum(x) = (-b / 16) * D0. Scales enter in f32 after a group's
//     instructions, so no weight is ever rounded.
//   - One instruction must stay inside a group. Its four lane groups hold the
//     four 32-element chunks, so for groups of 64 two, for groups of 32 four
//     lane-half swaps (v_permlane32_swap, v_permlane16_swap) exchange words
//     between the lane groups first.
//   - f32 activations are three bf16 parts (8 + 8 + 8 bits, exact) that
//     accumulate into one result.
// MI = 1 is for up to 4 tokens: token v is row 4v of the A operand, so each
// lane has one live result instead of four, and the scaling costs a quarter.
// MI = 4 takes 16 tokens. Each wave stages its own piece of x in LDS, in the
// element order that the unpacking gives the codes; no barrier until the join.
#include "common.hpp"
#include "kernels.hpp"

namespace mmk {

namespace {

constexpr int QThreads = 256;
constexpr int QWaves = QThreads / kWave;
constexpr int QStep = 128;  // elements of k in a step

template <class S>
struct __attribute__((packed, aligned(sizeof(S)))) QChunk {
    u32x4 v;
};

// Operand format of the codes and the activations.
struct CoreF16 {
    static constexpr uint32_t kSixteen = 0x4C004C00u;
    static constexpr uint32_t kMinusSixteen = 0xCC00CC00u;
    static constexpr int kShift = 6;  // the code's place in the mantissa of 16.0
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
struct CoreBF16 {
    static constexpr uint32_t kSixteen = 0x41804180u;
    static constexpr uint32_t kMinusSixteen = 0xC180C180u;
    static constexpr int kShift = 3;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <class T> struct CoreOf { using type = CoreBF16; };
template <> struct CoreOf<TF16> { using type = CoreF16; };

// Eight codes (nibble i = element i) to 16 + q in the order 0 4 1 5 2 6 3 7.
template <class C>
__device__ __forceinline__ u32x4 codes16(uint32_t w) {
    u32x4 r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int sh = 4 * p - C::kShift;
        const uint32_t t = sh >= 0 ? w >> (sh >= 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
        r[p] = (t & (0x000F000Fu << C::kShift)) | C::kSixteen;
    }
    return r;
}

// Eight activations as PARTS operand octets in that order.
template <class T>
__device__ __forceinline__ void stage_octet(const typename T::store_t* p, u32x4* out) {
    using S = typename T::store_t;
    if constexpr (T::code == 0) {
        const u32x4 v0 = reinterpret_cast<const QChunk<S>*>(p)->v;
        const u32x4 v1 = reinterpret_cast<const QChunk<S>*>(p + 4)->v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo = v0[i], hi = v1[i];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                out[q][i] = (lo >> 16) | (hi & 0xFFFF0000u);
                lo = __float_as_uint(__uint_as_float(lo) - __uint_as_float(lo & 0xFFFF0000u));
                hi = __float_as_uint(__uint_as_float(hi) - __uint_as_float(hi & 0xFFFF0000u));
            }
        }
    } else {
        const u32x4 v = reinterpret_cast<const QChunk<S>*>(p)->v;
        out[0][0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
        out[0][1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
        out[0][2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
        out[0][3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
    }
}

__device__ __forceinline__ float scale_value(uint16_t h, bool bf16) {
    return bf16 ? widen(TBF16{}, h) : widen(TF16{}, h);
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <class T, int GROUP, int MI, bool GATED>
__global__ __launch_bounds__(QThreads) void q4_rows(Q4Args a) {
    using S = typename T::store_t;
    using C = typename CoreOf<T>::type;
    constexpr int PARTS = T::code == 0 ? 3 : 1;
    constexpr int VT = MI == 1 ? 4 : 16;          // tokens of a pass
    constexpr int CS = MI == 1 ? 4 : PARTS == 3 ? 1 : 2;  // steps of a chunk
    constexpr int NT = GATED ? 2 : 1;             // tiles of 16 weight rows
    constexpr int GPS = QStep / GROUP;            // groups of a step
    constexpr int OCT = CS * QStep / 8;           // octets of a token's chunk
    constexpr int PITCH = OCT + 1;                // in 16-byte units; odd: banks
    __shared__ u32x4 xs[QWaves][PARTS][VT][PITCH];
    __shared__ float join[QWaves][NT][VT][17];
    __shared__ uint32_t s_scan[QWaves], s_found[3];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane & 15, c = lane >> 4;
    const uint32_t n0 = blockIdx.x * 16;
    const uint32_t tile = blockIdx.z * gridDim.y + blockIdx.y;
    if (tile >= a.tiles) return;
    const bool sbf = a.scale_dtype == 2;
    const uint32_t N = GATED ? 2 * a.n : a.n;
    const uint32_t G = a.k / GROUP;
    // This wave's steps of k.
    const uint32_t steps = (a.k + QStep - 1) / QStep;
    const uint32_t st0 = steps * wave / QWaves, st1 = steps * (wave + 1) / QWaves;

    // Where this block's rows come from.
    uint32_t expert = 0, row0 = 0, cnt = 0;
    if (a.mode == Q4_DENSE) {
        row0 = tile * VT;
        cnt = a.rows - row0 < VT ? a.rows - row0 : VT;
    } else if (a.mode == Q4_IDS) {
        row0 = tile;
        cnt = 1;
        expert = a.ids[row0];
    } else {
        // Tile number `tile` of the experts' row tiles: each thread counts the
        // tiles of its experts, a scan over the block places them.
        constexpr int EPT = 4;  // 1024 experts
        const uint32_t R = a.rows;
        uint32_t lo[EPT], tiles[EPT], mine = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const uint32_t e = threadIdx.x * EPT + i;
            uint32_t b = 0, d = 0;
            if (e < a.n_experts) { b = a.offsets[e]; d = a.offsets[e + 1]; }
            d = d < R ? d : R;
            lo[i] = b;
            tiles[i] = b < d ? (d - b + VT - 1) / VT : 0;
            mine += tiles[i];
        }
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const uint32_t v = (uint32_t)__shfl_up((int)upto, o, kWave);
            if (lane >= o) upto += v;
        }
        if (lane == kWave - 1) s_scan[wave] = upto;
        if (threadIdx.x == 0) s_found[2] = 0;
        __syncthreads();
        uint32_t at = upto - mine;
        for (int w = 0; w < wave; ++w) at += s_scan[w];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const uint32_t e = threadIdx.x * EPT + i;
            if (tile >= at && tile < at + tiles[i]) {
                const uint32_t b = lo[i] + (tile - at) * VT;
                uint32_t d = a.offsets[e + 1];
                d = d < R ? d : R;
                s_found[0] = e;
                s_found[1] = b;
                s_found[2] = d - b < VT ? d - b : VT;
            }
            at += tiles[i];
        }
        __syncthreads();
        expert = s_found[0];
        row0 = s_found[1];
        cnt = s_found[2];
        // Rows past the last expert's are zeros; the first tile's block writes them.
        if (tile == 0) {
            const uint32_t live = a.offsets[a.n_experts];
            for (uint64_t i = (uint64_t)live + threadIdx.x / 16; i < R; i += QThreads / 16) {
                if (n0 + (threadIdx.x & 15) < a.n)
                    static_cast<S*>(a.y)[i * a.ldy + n0 + (threadIdx.x & 15)] = 0;
            }
        }
        if (cnt == 0) return;
        expert = __builtin_amdgcn_readfirstlane(expert);
        row0 = __builtin_amdgcn_readfirstlane(row0);
        cnt = __builtin_amdgcn_readfirstlane(cnt);
    }
    S* const y = static_cast<S*>(a.y) + (int64_t)row0 * a.ldy;
    if (a.mode == Q4_IDS && expert >= a.n_experts) {
        if (threadIdx.x < 16 && n0 + threadIdx.x < a.n) y[n0 + threadIdx.x] = 0;
        return;
    }
    const S* const x = static_cast<const S*>(a.x) +
                       (int64_t)(a.mode == Q4_IDS ? row0 / a.x_div : row0) * a.ldx;

    // This lane's weight row in each tile; rows past n repeat the last and are not stored.
    const uint8_t* codes[NT];
    const uint16_t *sc[NT], *bi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t j = (n0 + r16 < a.n ? n0 + r16 : a.n - 1) + t * a.n;
        const uint64_t row = (uint64_t)expert * N + j;
        codes[t] = a.codes + row * (a.k / 2);
        sc[t] = a.scales + row * G;
        bi[t] = a.biases + row * G;
    }
    // The token whose activations this lane reads as row r16 of the A operand.
    const int tok = MI == 1 ? r16 >> 2 : r16;
    const u32x4(*const mine)[VT][PITCH] = xs[wave];
    const int vtok = tok < (int)cnt ? tok : (int)cnt - 1;

    f32x4 out[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) out[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 minus16 = {C::kMinusSixteen, C::kMinusSixteen, C::kMinusSixteen, C::kMinusSixteen};

    for (uint32_t s0 = st0; s0 < st1; s0 += CS) {
        // Codes of the chunk; chunks past the row's end read its start (their x is 0).
        u32x4 w[CS][NT];
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            const uint32_t k0 = (s0 + i) * QStep + c * 32;
            const bool in = s0 + i < st1 && k0 < a.k;
#pragma unroll
            for (int t = 0; t < NT; ++t) w[i][t] = ld16(codes[t] + (in ? k0 / 2 : 0));
        }
        // Activations of the chunk into LDS.
        for (uint32_t q = lane; q < cnt * OCT; q += kWave) {
            const uint32_t v = q / OCT, o = q % OCT;
            const uint32_t k0 = s0 * QStep + o * 8;
            u32x4 parts[PARTS];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) parts[p] = u32x4{0, 0, 0, 0};
            if (s0 + o / (QStep / 8) < st1 && k0 < a.k) stage_octet<T>(x + (int64_t)v * a.ldx + k0, parts);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) xs[wave][p][v][o] = parts[p];
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (s0 + i >= st1) break;
            // Words to instruction order: word g of lane group c then is octet oct(g, c).
            uint32_t cw[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int g = 0; g < 4; ++g) cw[t][g] = w[i][t][g];
                if constexpr (GROUP <= 64) {
                    swap32(cw[t][0], cw[t][2]);
                    swap32(cw[t][1], cw[t][3]);
                }
                if constexpr (GROUP == 32) {
                    swap16(cw[t][0], cw[t][1]);
                    swap16(cw[t][2], cw[t][3]);
                }
            }
#pragma unroll
            for (int gp = 0; gp < GPS; ++gp) {
                f32x4 d0 = {0.f, 0.f, 0.f, 0.f};
                f32x4 d[NT];
                u32x4 av[PARTS][4 / GPS];
#pragma unroll
                for (int j = 0; j < 4 / GPS; ++j) {
                    const int g = gp * (4 / GPS) + j;
                    const int oct = GROUP == 128 ? 4 * c + g
                                    : GROUP == 64 ? 8 * (g >> 1) + 4 * (c & 1) + 2 * (c >> 1) + (g & 1)
                                                  : 4 * g + c;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        av[p][j] = mine[p][vtok][i * (QStep / 8) + oct];
                        d0 = C::mma(av[p][j], minus16, d0);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    d[t] = d0;
#pragma unroll
                    for (int j = 0; j < 4 / GPS; ++j) {
                        const u32x4 bq = codes16<C>(cw[t][gp * (4 / GPS) + j]);
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) d[t] = C::mma(av[p][j], bq, d[t]);
                    }
                    const uint32_t g0 = (s0 + i) * GPS + gp;
                    const uint32_t gi = g0 < G ? g0 : G - 1;
                    const float s = scale_value(sc[t][gi], sbf);
                    const float b = scale_value(bi[t][gi], sbf) * -0.0625f;
#pragma unroll
                    for (int v = 0; v < MI; ++v)
                        out[t][v] = __builtin_fmaf(b, d0[v], __builtin_fmaf(s, d[t][v], out[t][v]));
                }
            }
        }
        // The next chunk overwrites what this one reads.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }

    // Join the four pieces of k.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < MI; ++v) join[wave][t][MI == 1 ? c : 4 * c + v][r16] = out[t][v];
    __syncthreads();
    const uint32_t v = threadIdx.x / 16, j = threadIdx.x & 15;
    if (v < cnt && n0 + j < a.n) {
        float sum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sum[t] = join[0][t][v][j];
#pragma unroll
            for (int w = 1; w < QWaves; ++w) sum[t] += join[w][t][v][j];
        }
        float r = sum[0];
        if constexpr (GATED) r = sum[0] / (1.f + expf(-sum[0])) * sum[1];
        y[(int64_t)v * a.ldy + n0 + j] = narrow(T{}, r);
    }
}

template <class T, int GROUP>
const void* pick(bool wide, bool gated) {
    if (wide) return gated ? (const void*)&q4_rows<T, GROUP, 4, true> : (const void*)&q4_rows<T, GROUP, 4, false>;
    return gated ? (const void*)&q4_rows<T, GROUP, 1, true> : (const void*)&q4_rows<T, GROUP, 1, false>;
}
template <class T>
const void* pick(uint32_t group, bool wide, bool gated) {
    return group == 32 ? pick<T, 32>(wide, gated) : group == 64 ? pick<T, 64>(wide, gated) : pick<T, 128>(wide, gated);
}

}  // namespace

hipError_t launch_q4(const Q4Args& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_Q4;
    // Sixteen tokens a pass where an expert has more than 4 rows on average.
    const bool wide = a.mode == Q4_DENSE ? a.rows > 4 : a.mode == Q4_SORTED && a.rows > 4ull * a.n_experts;
    const uint32_t vt = wide ? 16 : 4;
    L->variant = (int)vt;
    uint64_t tiles = a.rows;
    if (a.mode == Q4_DENSE) tiles = (a.rows + vt - 1) / vt;
    // Sorted: every expert with rows may end inside a tile.
    if (a.mode == Q4_SORTED) tiles = a.rows / vt + (a.rows < a.n_experts ? a.rows : a.n_experts);
    const void* fn = a.dtype == 0   ? pick<TF32>(a.group, wide, a.gated)
                     : a.dtype == 1 ? pick<TF16>(a.group, wide, a.gated)
                                    : pick<TBF16>(a.group, wide, a.gated);
    Q4Args b = a;
    b.tiles = (uint32_t)tiles;
    const uint32_t gy = (uint32_t)(tiles < 32768 ? tiles : 32768);
    void* args[] = {&b};
    return hipLaunchKernel(fn, dim3((a.n + 15) / 16, gy, (uint32_t)((tiles + gy - 1) / gy)),
                           dim3(QThreads), args, 0, s);
}

}  // namespace mmk
