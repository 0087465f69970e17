// Products with 4-bit weights and group scales, y = sum over groups of
// s * (q . x) + b * sum(x), on matrix instructions.
//
// A wave takes TN tiles of 16 rows of W and a contiguous piece of k, 128
// elements (64 bytes of codes a row) at a step: lane l loads the 16 bytes at
// chunk l / 16 of row l % 16. The W waves of a block take the pieces of k and
// join their sums through LDS. The codes are the B operand of
// v_mfma_f32_16x16x32 (column = row of W), the activations the A operand (row =
// token):
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
// The loads of the next chunk (activations, codes, scales) are issued before
// the current one is computed.
#include "common.hpp"
#include "kernels.hpp"

namespace mmk {

namespace {

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

// Eight activations as operand octets in that order: one, or for f32 three
// bf16 parts (each the rest's upper 16 bits, which is exact).
template <class T>
__device__ __forceinline__ void octet(const u32x4* in, u32x4* out) {
    if constexpr (T::code == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo = in[0][i], hi = in[1][i];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                out[q][i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
                lo = __float_as_uint(__uint_as_float(lo) - __uint_as_float(lo & 0xFFFF0000u));
                hi = __float_as_uint(__uint_as_float(hi) - __uint_as_float(hi & 0xFFFF0000u));
            }
        }
    } else {
        const u32x4 v = in[0];
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

// NV neighbouring 16-bit values at a 2-byte aligned address, two to a register.
template <int NV>
__device__ __forceinline__ void load_pairs(const uint16_t* p, uint32_t* r) {
    struct __attribute__((packed, aligned(2))) D { uint32_t v; };
    struct __attribute__((packed, aligned(2))) D2 { u32x2 v; };
    if constexpr (NV == 1) {
        r[0] = p[0];
    } else if constexpr (NV == 2) {
        r[0] = reinterpret_cast<const D*>(p)->v;
    } else if constexpr (NV == 4) {
        const u32x2 v = reinterpret_cast<const D2*>(p)->v;
        r[0] = v[0];
        r[1] = v[1];
    } else {
#pragma unroll
        for (int i = 0; i < NV / 8; ++i) {
            const u32x4 v = reinterpret_cast<const QChunk<uint16_t>*>(p + 8 * i)->v;
#pragma unroll
            for (int j = 0; j < 4; ++j) r[4 * i + j] = v[j];
        }
    }
}

// Row tile `tile` of sorted rows: its expert, first row and row count (0: none).
// Every wave walks the experts' tile counts, 64 experts at a time.
template <int VT>
__device__ __forceinline__ void find_tile(const Q4Args& a, uint32_t tile, int lane, uint32_t* expert,
                                          uint32_t* row0, uint32_t* cnt) {
    uint32_t before = 0;
    for (uint32_t e0 = 0; e0 < a.n_experts; e0 += kWave) {
        const uint32_t e = e0 + lane;
        uint32_t lo = 0, hi = 0;
        if (e < a.n_experts) {
            lo = a.offsets[e];
            hi = a.offsets[e + 1];
        }
        hi = hi < a.rows ? hi : a.rows;
        const uint32_t n = lo < hi ? (hi - lo + VT - 1) / VT : 0;
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const uint32_t v = (uint32_t)__shfl_up((int)upto, o, kWave);
            if (lane >= o) upto += v;
        }
        const uint64_t past = __ballot(tile < before + upto);
        if (past) {
            const int f = __ffsll((unsigned long long)past) - 1;
            const uint32_t first = lo + (tile - (before + upto - n)) * VT;
            *expert = e0 + f;
            *row0 = (uint32_t)__builtin_amdgcn_readlane((int)first, f);
            const uint32_t end = (uint32_t)__builtin_amdgcn_readlane((int)hi, f);
            *cnt = end - *row0 < VT ? end - *row0 : VT;
            return;
        }
        before += (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
    }
    *cnt = 0;
}

template <class T, int GROUP, int MI, bool GATED, int TN, int W>
__global__ __launch_bounds__(W* kWave) void q4_rows(Q4Args a) {
    using S = typename T::store_t;
    using C = typename CoreOf<T>::type;
    constexpr int PARTS = T::code == 0 ? 3 : 1;
    constexpr int VT = MI == 1 ? 4 : 16;                                        // tokens of a pass
    constexpr int CS = MI == 1 ? (PARTS == 3 ? 2 : 4) : (PARTS == 3 ? 1 : 2);   // steps of a chunk
    constexpr int NT = GATED ? 2 * TN : TN;       // tiles of 16 weight rows
    constexpr int GPS = QStep / GROUP;            // groups of a step
    constexpr int NV = CS * GPS;                  // groups of a chunk
    constexpr int SR = NV == 1 ? 1 : NV / 2;      // registers of their scales
    constexpr int OCT = CS * QStep / 8;           // octets of a token's chunk
    constexpr int XL = VT * OCT / kWave;          // octets a lane stages
    constexpr int PITCH = OCT + 1;                // in 16-byte units; odd: banks
    __shared__ u32x4 xs[W][PARTS][VT][PITCH];
    __shared__ float join[W][NT][VT][17];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r16 = lane & 15, c = lane >> 4;
    const uint32_t n0 = blockIdx.x * (16 * TN);
    const uint32_t tile = blockIdx.z * gridDim.y + blockIdx.y;
    if (tile >= a.tiles) return;
    const bool sbf = a.scale_dtype == 2;
    const uint32_t N = GATED ? 2 * a.n : a.n;
    const uint32_t G = a.k / GROUP;
    // This wave's steps of k.
    const uint32_t steps = (a.k + QStep - 1) / QStep;
    const uint32_t st0 = steps * wave / W, st1 = steps * (wave + 1) / W;

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
        find_tile<VT>(a, tile, lane, &expert, &row0, &cnt);
        // Rows past the last expert's are zeros; the first tile's block writes them.
        if (tile == 0) {
            const uint32_t live = a.offsets[a.n_experts];
            for (uint64_t i = (uint64_t)live + wave; i < a.rows; i += W) {
                if (lane < 16 * TN && n0 + lane < a.n) static_cast<S*>(a.y)[i * a.ldy + n0 + lane] = 0;
            }
        }
        if (cnt == 0) return;
    }
    S* const y = static_cast<S*>(a.y) + (int64_t)row0 * a.ldy;
    if (a.mode == Q4_IDS && expert >= a.n_experts) {
        if (threadIdx.x < 16 * TN && n0 + threadIdx.x < a.n) y[n0 + threadIdx.x] = 0;
        return;
    }
    const S* const x = static_cast<const S*>(a.x) +
                       (int64_t)(a.mode == Q4_IDS ? row0 / a.x_div : row0) * a.ldx;

    // This lane's weight row in each tile (gate tiles, then up tiles); rows past
    // n repeat the last and are not stored.
    const uint8_t* codes[NT];
    const uint16_t *sc[NT], *bi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t j0 = n0 + (t % TN) * 16 + r16;
        const uint32_t j = (j0 < a.n ? j0 : a.n - 1) + (t / TN) * a.n;
        const uint64_t row = (uint64_t)expert * N + j;
        codes[t] = a.codes + row * (a.k / 2);
        sc[t] = a.scales + row * G;
        bi[t] = a.biases + row * G;
    }
    // The token whose activations this lane reads as row r16 of the A operand;
    // rows past the last token repeat it and are not stored.
    const int tok = MI == 1 ? r16 >> 2 : r16;
    const int vtok = tok < (int)cnt ? tok : (int)cnt - 1;

    struct Chunk {
        u32x4 x[XL][PARTS == 3 ? 2 : 1];
        u32x4 w[CS][NT];
        uint32_t s[NT][SR], b[NT][SR];
    };
    const auto load = [&](Chunk& q, uint32_t s0) {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const uint32_t v = (i * kWave + lane) / OCT, o = (i * kWave + lane) % OCT;
            const uint32_t k0 = s0 * QStep + o * 8;
#pragma unroll
            for (int p = 0; p < (PARTS == 3 ? 2 : 1); ++p) {
                q.x[i][p] = u32x4{0, 0, 0, 0};
                if (v < cnt && s0 + o / (QStep / 8) < st1 && k0 < a.k)
                    q.x[i][p] = reinterpret_cast<const QChunk<S>*>(x + (int64_t)v * a.ldx + k0 + 4 * p)->v;
            }
        }
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (s0 + i >= st1) break;
            // Chunks past the row's end read its start: their activations are 0.
            const uint32_t k0 = (s0 + i) * QStep + c * 32;
#pragma unroll
            for (int t = 0; t < NT; ++t) q.w[i][t] = ld16(codes[t] + (k0 < a.k ? k0 / 2 : 0));
        }
        const uint32_t g0 = s0 * GPS;
        if (g0 + NV <= G) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                load_pairs<NV>(sc[t] + g0, q.s[t]);
                load_pairs<NV>(bi[t] + g0, q.b[t]);
            }
        } else {  // the row's last chunk, cut short
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < SR; ++i) {
                    const uint32_t e0 = g0 + 2 * i < G ? g0 + 2 * i : G - 1;
                    const uint32_t e1 = g0 + 2 * i + 1 < G ? g0 + 2 * i + 1 : G - 1;
                    q.s[t][i] = sc[t][e0] | ((uint32_t)sc[t][e1] << 16);
                    q.b[t][i] = bi[t][e0] | ((uint32_t)bi[t][e1] << 16);
                }
        }
    };

    f32x4 out[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) out[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 minus16 = {C::kMinusSixteen, C::kMinusSixteen, C::kMinusSixteen, C::kMinusSixteen};

    Chunk cur;
    if (st0 < st1) load(cur, st0);
    for (uint32_t s0 = st0; s0 < st1; s0 += CS) {
        // Activations of the chunk into LDS.
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const uint32_t v = (i * kWave + lane) / OCT, o = (i * kWave + lane) % OCT;
            u32x4 parts[PARTS];
            octet<T>(cur.x[i], parts);
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                if (v < cnt) xs[wave][p][v][o] = parts[p];
        }
        Chunk nxt;
        if (s0 + CS < st1) load(nxt, s0 + CS);
        // One wave writes and reads its LDS in order: only the compiler needs telling.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (s0 + i >= st1) break;
            // Words to instruction order.
            uint32_t cw[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int g = 0; g < 4; ++g) cw[t][g] = cur.w[i][t][g];
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
                u32x4 av[PARTS][4 / GPS];
#pragma unroll
                for (int j = 0; j < 4 / GPS; ++j) {
                    // Word g of lane group c is octet oct of the step.
                    const int g = gp * (4 / GPS) + j;
                    const int oct = GROUP == 128  ? 4 * c + g
                                    : GROUP == 64 ? 8 * (g >> 1) + 4 * (c & 1) + 2 * (c >> 1) + (g & 1)
                                                  : 4 * g + c;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        av[p][j] = xs[wave][p][vtok][i * (QStep / 8) + oct];
                        d0 = C::mma(av[p][j], minus16, d0);
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4 d = d0;
#pragma unroll
                    for (int j = 0; j < 4 / GPS; ++j) {
                        const u32x4 bq = codes16<C>(cw[t][gp * (4 / GPS) + j]);
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) d = C::mma(av[p][j], bq, d);
                    }
                    const int gi = i * GPS + gp;
                    const uint16_t sh = (uint16_t)(cur.s[t][gi / 2] >> (16 * (gi & 1)));
                    const uint16_t bh = (uint16_t)(cur.b[t][gi / 2] >> (16 * (gi & 1)));
                    const float sv = scale_value(sh, sbf);
                    const float bv = scale_value(bh, sbf) * -0.0625f;
#pragma unroll
                    for (int v = 0; v < MI; ++v)
                        out[t][v] = __builtin_fmaf(bv, d0[v], __builtin_fmaf(sv, d[v], out[t][v]));
                }
            }
        }
        // The next chunk overwrites what this one reads.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        cur = nxt;
    }

    // Join the W pieces of k.
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < MI; ++v) join[wave][t][MI == 1 ? c : 4 * c + v][r16] = out[t][v];
    __syncthreads();
    for (uint32_t q = threadIdx.x; q < VT * 16 * TN; q += W * kWave) {
        const uint32_t v = q / (16 * TN), tt = q / 16 % TN, j = q % 16;
        const uint32_t col = n0 + tt * 16 + j;
        if (v >= cnt || col >= a.n) continue;
        float sum[GATED ? 2 : 1];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            sum[h] = join[0][h * TN + tt][v][j];
#pragma unroll
            for (int w = 1; w < W; ++w) sum[h] += join[w][h * TN + tt][v][j];
        }
        float r = sum[0];
        if constexpr (GATED) r = sum[0] / (1.f + expf(-sum[0])) * sum[1];
        y[(int64_t)v * a.ldy + col] = narrow(T{}, r);
    }
}

// The instances: up to 4 tokens a pass on one tile; 16 on one tile (eight
// pieces of k, for few blocks) or on 64 weight rows (staging x costs less).
enum Form { NARROW, WIDE_FEW, WIDE };
template <class T, int GROUP, bool GATED>
const void* pick(Form f) {
    switch (f) {
        case NARROW: return (const void*)&q4_rows<T, GROUP, 1, GATED, 1, 4>;
        case WIDE_FEW: return (const void*)&q4_rows<T, GROUP, 4, GATED, 1, 8>;
        default: return (const void*)&q4_rows<T, GROUP, 4, GATED, GATED ? 2 : 4, 4>;
    }
}
template <class T, int GROUP>
const void* pick(Form f, bool gated) {
    return gated ? pick<T, GROUP, true>(f) : pick<T, GROUP, false>(f);
}
template <class T>
const void* pick(uint32_t group, Form f, bool gated) {
    return group == 32 ? pick<T, 32>(f, gated) : group == 64 ? pick<T, 64>(f, gated) : pick<T, 128>(f, gated);
}

}  // namespace

hipError_t launch_q4(const Q4Args& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_Q4;
    // Sixteen tokens a pass where an expert has more than 4 rows on average.
    const bool wide = a.mode == Q4_DENSE ? a.rows > 4 : a.mode == Q4_SORTED && a.rows > 4ull * a.n_experts;
    const uint32_t vt = wide ? 16 : 4;
    uint64_t tiles = a.rows;
    if (a.mode == Q4_DENSE) tiles = (a.rows + vt - 1) / vt;
    // Sorted: every expert with rows may end inside a tile.
    if (a.mode == Q4_SORTED) tiles = a.rows / vt + (a.rows < a.n_experts ? a.rows : a.n_experts);
    Form f = NARROW;
    uint32_t tn = 1, w = 4;
    if (wide) {
        tn = a.gated ? 2 : 4;
        f = WIDE;
        if (tiles * ((a.n + 16 * tn - 1) / (16 * tn)) < 512) {
            f = WIDE_FEW;
            tn = 1;
            w = 8;
        }
    }
    L->variant = (int)(vt + 256 * tn);
    const void* fn = a.dtype == 0   ? pick<TF32>(a.group, f, a.gated)
                     : a.dtype == 1 ? pick<TF16>(a.group, f, a.gated)
                                    : pick<TBF16>(a.group, f, a.gated);
    Q4Args b = a;
    b.tiles = (uint32_t)tiles;
    const uint32_t gy = (uint32_t)(tiles < 32768 ? tiles : 32768);
    void* args[] = {&b};
    return hipLaunchKernel(fn, dim3((a.n + 16 * tn - 1) / (16 * tn), gy, (uint32_t)((tiles + gy - 1) / gy)),
                           dim3(w * kWave), args, 0, s);
}

}  // namespace mmk
