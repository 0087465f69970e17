// Products with 4-bit weights and group scales, y = sum over groups of
// s * (q . x) + b * sum(x), on matrix instructions.
//
// A wave reads tiles of 16 rows of W, 128 elements of k (64 bytes of codes a
// row) at a step: lane l loads the 16 bytes at chunk l / 16 of row l % 16. The
// codes are the B operand of v_mfma_f32_16x16x32 (column = row of W), the
// activations the A operand (row = token):
//   - A code becomes an operand by placing its four bits in the mantissa of
//     1.0, which is 1 + q / 16, exact in f16 and bf16: one shift and one
//     and-or for two codes, no conversion. The accumulator starts at minus the
//     group's sum of x and so ends at q . x / 16 (the 1 taken back after the
//     instructions instead, by a coefficient b - 16 s, had 1.5 times the error);
//     outputs are multiplied by 16. The accumulator stays below 2^128 on the way
//     for every group and |x| < 2^120 (in the mantissa of 16.0 the same sums
//     passed 2^128 from |x| = 2^116 on).
//     The sum is taken where x is staged, or, for 16 tokens of 16 bits, by the
//     same instruction with a constant operand (staging 31 -> 10 instructions
//     an octet). Scales enter in f32 after a group's instructions, so no weight
//     is ever rounded.
//   - f32 activations are three bf16 parts (8 + 8 + 8 bits, exact down to
//     2^-133). The upper parts have an accumulator and a sum of their own: their
//     products and sums are short enough to be nearly exact in f32, and the lower
//     parts' roundings are small (error against 64 bits 4e-8 to 4e-7 of the result
//     in norm, by k and group; 2e-7 where one accumulator and one sum had 5e-7 to
//     1.5e-6).
//   - A sum must not leave its group. The four lane groups of an instruction
//     hold the step's four 32-element chunks. With up to 4 tokens (MI = 1) the A
//     operand has 16 rows for 4 tokens: row 4v + g holds token v in lane group g
//     and zeros in the others, so the four results of a lane are the four
//     chunks' sums. With 16 tokens (MI = 4) lane-half swaps
//     (v_permlane32_swap, v_permlane16_swap) first exchange words between the
//     lane groups, two for groups of 64, four for groups of 32.
//
// q4_split (few blocks): the W waves of a block take pieces of k for the same
// rows, each stages its own piece of x in LDS, and the sums are joined there;
// no barrier until then. q4_block (many rows and tokens): the waves take
// different rows of W and share x, staged a chunk of k at a time in two buffers,
// one barrier a chunk. Both issue the loads of the next chunk before computing
// the current one.
//
// Measured (kernel alone): one token, 11008 x 4096 f16, groups of 128: 8.3 us, 2.9
// TB/s; one token's eight gated experts of 1408 x 2048, bf16, groups of 32: 10.3 us,
// 2.8 TB/s; both a launch, one or two memory round trips and 2 to 3 us of vector
// issue. 512 f32 rows over 64 experts of 2048 x 1408, groups of 64: 47 us, 2.4 TB/s,
// bound by vector issue (19 us) and matrix instructions (8 us) between barriers. A
// stream of the same bytes in this access pattern reaches 5.1 TB/s.
#include <type_traits>

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
    static constexpr uint32_t kOne = 0x3C003C00u;
    static constexpr uint32_t kMinusOne = 0xBC00BC00u;
    static constexpr int kShift = 6;  // the code's place in the mantissa of 1.0
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
struct CoreBF16 {
    static constexpr uint32_t kOne = 0x3F803F80u;
    static constexpr uint32_t kMinusOne = 0xBF80BF80u;
    static constexpr int kShift = 3;
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <class T> struct CoreOf { using type = CoreBF16; };
template <> struct CoreOf<TF16> { using type = CoreF16; };

// Eight codes (nibble i = element i) to 1 + q / 16 in the order 0 4 1 5 2 6 3 7.
// The mask is a scalar, the 1.0s a vector register: as literals they would not
// fit one and-or.
template <class C>
__device__ __forceinline__ u32x4 codes16(uint32_t w, uint32_t mask, uint32_t one) {
    u32x4 r;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int sh = 4 * p - C::kShift;
        const uint32_t t = sh >= 0 ? w >> (sh >= 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
        r[p] = (t & mask) | one;
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

// Inclusive sum over the lanes up to this one: within rows of 16 lanes, then
// each row's last lane onto the rows after it.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    int x = (int)v;
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);  // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);  // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);  // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return (uint32_t)x;
}

// Row tile `tile` of sorted rows: its expert, first row and row count. Past the
// experts' tiles: a row count of 0, and in row0 the tiles past them.
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
        const uint32_t upto = wave_scan(n);
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
    *row0 = tile - before;
    *cnt = 0;
}

// The rows of x and y that a block takes, and their expert. A block without
// rows (or whose rows have no expert: written as zeros here) has cnt = 0.
struct Rows {
    uint32_t expert, row0, cnt;
};
// VT: tokens of a tile; COLS: output columns of a block of THREADS, from n0 on.
template <class S, int VT, int COLS, int THREADS>
__device__ __forceinline__ Rows block_rows(const Q4Args& a, uint32_t n0) {
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t tile = blockIdx.z * gridDim.y + blockIdx.y;
    Rows r{0, 0, 0};
    if (tile >= a.tiles) return r;
    S* const y = static_cast<S*>(a.y);
    if (a.mode == Q4_DENSE) {
        r.row0 = tile * VT;
        r.cnt = a.rows - r.row0 < VT ? a.rows - r.row0 : VT;
    } else if (a.mode == Q4_IDS) {
        r.row0 = tile;
        r.expert = a.ids[tile];
        r.cnt = r.expert < a.n_experts;
        if (!r.cnt) {
            for (uint32_t j = threadIdx.x; j < COLS; j += THREADS)
                if (n0 + j < a.n) y[(int64_t)tile * a.ldy + n0 + j] = 0;
        }
    } else {
        find_tile<VT>(a, tile, lane, &r.expert, &r.row0, &r.cnt);
        // Rows past the last expert's are zeros, VT of them for each tile past the
        // experts' own (65536 rows of 256 x 256, half of them without an expert:
        // 1048 us where the first tile wrote them all, 34 us so; all with: 49 us).
        if (r.cnt == 0) {
            const uint64_t z0 = a.offsets[a.n_experts] + (uint64_t)r.row0 * VT;
            for (uint32_t q = threadIdx.x; q < VT * COLS; q += THREADS) {
                const uint64_t i = z0 + q / COLS;
                const uint32_t j = n0 + q % COLS;
                if (i < a.rows && j < a.n) y[i * a.ldy + j] = 0;
            }
        }
    }
    return r;
}

// Sum of eight values a lane over the GROUP / 8 lanes that hold a group.
template <int GROUP>
__device__ __forceinline__ float group_sum(const float (&f)[8]) {
    float v = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    const auto from = [&](auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
            0, (int)__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v += from(std::integral_constant<int, 0xB1>{});   // quad_perm 1 0 3 2
    v += from(std::integral_constant<int, 0x4E>{});   // quad_perm 2 3 0 1
    if constexpr (GROUP >= 64) v += from(std::integral_constant<int, 0x141>{});   // row_half_mirror
    if constexpr (GROUP >= 128) v += from(std::integral_constant<int, 0x140>{});  // row_mirror
    return v;
}

// Sums of NT tiles of 16 weight rows over a range of k: the operands' places,
// the loads of a chunk of CS steps, and its arithmetic.
template <class T, class ST, int GROUP, int MI, int NT, int CS>
struct Tiles {
    using S = typename T::store_t;
    using C = typename CoreOf<T>::type;
    static constexpr int PARTS = T::code == 0 ? 3 : 1;
    static constexpr int SUMS = T::code == 0 ? 2 : 1;
    static constexpr bool STAGED_SUMS = MI == 1 || PARTS > 1;
    static constexpr int VT = MI == 1 ? 4 : 16;             // tokens
    static constexpr bool MASKED = MI == 1 && GROUP < QStep;
    static constexpr int ROWS = MASKED ? VT + 1 : VT;       // staged rows: a last one of zeros
    static constexpr int GPS = QStep / GROUP;               // groups of a step
    static constexpr int NV = CS * GPS;                     // groups of a chunk
    static constexpr int SR = NV == 1 ? 1 : NV / 2;         // registers of their scales
    static constexpr int OCT = CS * QStep / 8;              // octets of a token's chunk
    static constexpr int PITCH = OCT + 1;                   // in 16-byte units; odd: banks
    static constexpr int XR = PARTS == 3 ? 2 : 1;           // 16-byte loads of an octet
    struct Stage {
        u32x4 x[PARTS][ROWS][PITCH];
        // Minus each token's sum of a group; MI = 1: a token's groups together.
        // f32: of the upper parts, and of the rest.
        __attribute__((aligned(16))) float sum[SUMS][MI == 1 ? VT : NV][MI == 1 ? NV : VT];
    };

    struct Codes {
        u32x4 w[CS][NT];
        uint32_t s[NT][SR], b[NT][SR];
    };

    const uint8_t* codes[NT];      // first row of each tile, the same for the wave
    const uint16_t *sc[NT], *bi[NT];
    uint32_t coff[NT], goff[NT];   // this lane's row and chunk from there
    f32x4 out[NT];                 // sixteenths of the sums; MI = 1: out[t][0] alone
    uint32_t k, groups, mask, one;
    int c, xrow;

    // j[t]: first row of tile t; rows past `end` repeat the last and are not stored.
    __device__ __forceinline__ void init(const Q4Args& a, uint64_t expert_row, const uint32_t (&j)[NT],
                                         const uint32_t (&end)[NT], int lane, uint32_t cnt) {
        k = a.k;
        groups = k / GROUP;
        c = lane >> 4;
        const int r16 = lane & 15;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t j0 = j[t] < end[t] ? j[t] : end[t] - 1;
            const uint32_t r = r16 < (int)(end[t] - j0) ? r16 : end[t] - j0 - 1;
            codes[t] = a.codes + (expert_row + j0) * (k / 2);
            sc[t] = a.scales + (expert_row + j0) * groups;
            bi[t] = a.biases + (expert_row + j0) * groups;
            coff[t] = r * (k / 2) + c * 16;
            goff[t] = r * groups;
            out[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        // The staged row that is this lane's row of the A operand; rows past the
        // last token repeat it and are not stored.
        const int tok = MI == 1 ? r16 >> 2 : r16;
        xrow = tok < (int)cnt ? tok : (int)cnt - 1;
        if (MASKED && (r16 & 3) != c) xrow = VT;
        mask = 0x000F000Fu << C::kShift;
        one = C::kOne;
        asm volatile("" : "+s"(mask), "+v"(one));
    }

    // Scales first, codes by step: a step is computed as soon as its own have arrived.
    __device__ __forceinline__ void load(Codes& q, uint32_t s0, uint32_t st1) const {
        const uint32_t g0 = s0 * GPS;
        if (g0 + NV <= groups) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                load_pairs<NV>(sc[t] + (goff[t] + g0), q.s[t]);
                load_pairs<NV>(bi[t] + (goff[t] + g0), q.b[t]);
            }
        } else {  // the row's last chunk, cut short
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < SR; ++i) {
                    const uint32_t e0 = goff[t] + (g0 + 2 * i < groups ? g0 + 2 * i : groups - 1);
                    const uint32_t e1 = goff[t] + (g0 + 2 * i + 1 < groups ? g0 + 2 * i + 1 : groups - 1);
                    q.s[t][i] = sc[t][e0] | ((uint32_t)sc[t][e1] << 16);
                    q.b[t][i] = bi[t][e0] | ((uint32_t)bi[t][e1] << 16);
                }
        }
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (s0 + i >= st1) break;
            // Chunks past the row's end read its start: their activations are 0.
            const uint32_t k0 = (s0 + i) * QStep;
            const bool in = k0 + c * 32 < k;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t off = coff[t] + k0 / 2;
                if (k0 + QStep > k) off = in ? off : coff[t] - c * 16;
                q.w[i][t] = ld16(codes[t] + off);
            }
        }
    }

    // Octet `o` of token v's chunk from s0 on; past the row's end, another of the row.
    __device__ __forceinline__ void load_x(u32x4 (&q)[XR], const char* x, uint32_t v, uint32_t ldx,
                                           uint32_t s0, uint32_t o) const {
        const uint32_t k0 = s0 * QStep + o * 8 < k ? s0 * QStep + o * 8 : 0;
        const uint32_t at = (v * ldx + k0) * sizeof(S);
#pragma unroll
        for (int p = 0; p < XR; ++p) q[p] = reinterpret_cast<const QChunk<S>*>(x + (at + 16 * p))->v;
    }
    // Its place in LDS; zeros past the row's end.
    __device__ __forceinline__ void stage(Stage& xs, u32x4 (&q)[XR], uint32_t v, uint32_t s0,
                                          uint32_t o) const {
        if ((s0 + CS) * QStep > k && s0 * QStep + o * 8 >= k) {
#pragma unroll
            for (int p = 0; p < XR; ++p) q[p] = u32x4{0, 0, 0, 0};
        }
        u32x4 parts[PARTS];
        octet<T>(q, parts);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) xs.x[p][v][o] = parts[p];
        // The lanes of 16 neighbouring octets hold one token: whole rows of lanes are here.
        if constexpr (!STAGED_SUMS) return;
        float f[SUMS][8];
        if constexpr (T::code == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = q[i / 4][i % 4];
                f[0][i] = __uint_as_float(bits & 0xFFFF0000u);
                f[SUMS - 1][i] = __uint_as_float(bits) - f[0][i];
            }
        } else {
            unpack8(T{}, q[0], f[0]);
        }
        const uint32_t g = o / (GROUP / 8);
#pragma unroll
        for (int h = 0; h < SUMS; ++h) {
            const float sum = group_sum<GROUP>(f[h]);
            if (o % (GROUP / 8) == 0) xs.sum[h][MI == 1 ? v : g][MI == 1 ? g : v] = -sum;
        }
    }

    __device__ __forceinline__ void compute(const Codes& q, const Stage& xs, uint32_t s0, uint32_t st1) {
        // Accumulators that one chain of instructions fills; groups of those.
        constexpr int CHAINS = MI == 1 ? 1 : GPS, PER = 4 / CHAINS;
#pragma unroll
        for (int i = 0; i < CS; ++i) {
            if (s0 + i >= st1) break;
            uint32_t cw[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int g = 0; g < 4; ++g) cw[t][g] = q.w[i][t][g];
                if constexpr (MI > 1 && GROUP <= 64) {
                    swap32(cw[t][0], cw[t][2]);
                    swap32(cw[t][1], cw[t][3]);
                }
                if constexpr (MI > 1 && GROUP == 32) {
                    swap16(cw[t][0], cw[t][1]);
                    swap16(cw[t][2], cw[t][3]);
                }
            }
#pragma unroll
            for (int gp = 0; gp < CHAINS; ++gp) {
                u32x4 av[PARTS][PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    // Word g of lane group c is octet oct of the step.
                    const int g = gp * PER + j;
                    const int oct = MI == 1 || GROUP == 128 ? 4 * c + g
                                    : GROUP == 64 ? 8 * (g >> 1) + 4 * (c & 1) + 2 * (c >> 1) + (g & 1)
                                                  : 4 * g + c;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) av[p][j] = xs.x[p][xrow][i * (QStep / 8) + oct];
                }
                // -sum(x) of each group (MI = 1) or token: by parts, and whole.
                float sums[SUMS][4], sum[4];
                if constexpr (STAGED_SUMS) {
#pragma unroll
                    for (int h = 0; h < SUMS; ++h)
#pragma unroll
                        for (int v = 0; v < (MI == 1 ? GPS : 4); ++v)
                            sums[h][v] = MI == 1 ? xs.sum[h][c][i * GPS + v] : xs.sum[h][i * GPS + gp][4 * c + v];
                } else {
                    const u32x4 m1 = {C::kMinusOne, C::kMinusOne, C::kMinusOne, C::kMinusOne};
                    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < PER; ++j) d = C::mma(av[0][j], m1, d);
#pragma unroll
                    for (int v = 0; v < 4; ++v) sums[0][v] = d[v];
                }
#pragma unroll
                for (int v = 0; v < (MI == 1 ? GPS : 4); ++v)
                    sum[v] = SUMS == 1 ? sums[0][v] : sums[0][v] + sums[SUMS - 1][v];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4 acc[SUMS];
#pragma unroll
                    for (int h = 0; h < SUMS; ++h) {
                        // MI = 1: result i starts a group or continues it (two chunks of 64).
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            acc[h][v] = MI > 1               ? sums[h][v]
                                        : v % (4 / GPS) == 0 ? sums[h][v / (4 / GPS)]
                                                             : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const u32x4 bq = codes16<C>(cw[t][gp * PER + j], mask, one);
                        acc[0] = C::mma(av[0][j], bq, acc[0]);
#pragma unroll
                        for (int p = 1; p < PARTS; ++p) acc[SUMS - 1] = C::mma(av[p][j], bq, acc[SUMS - 1]);
                    }
                    f32x4 d = acc[0];
                    if constexpr (SUMS > 1) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) d[v] += acc[1][v];
                    }
                    // MI = 1: results 0..3 are the step's chunks (one value without
                    // the mask); MI = 4: four tokens of one group.
#pragma unroll
                    for (int h = 0; h < GPS / CHAINS; ++h) {
                        const int gi = i * GPS + gp + h;
                        const float sv = widen(ST{}, (uint16_t)(q.s[t][gi / 2] >> (16 * (gi & 1))));
                        const float bv = widen(ST{}, (uint16_t)(q.b[t][gi / 2] >> (16 * (gi & 1))));
                        const float b16 = bv * -0.0625f;  // of -sum(x), in sixteenths
                        if constexpr (MI == 1) {
                            const float dv = GROUP == 64 ? d[2 * h] + d[2 * h + 1] : d[h];
                            out[t][0] = __builtin_fmaf(b16, sum[h], __builtin_fmaf(sv, dv, out[t][0]));
                        } else {
#pragma unroll
                            for (int v = 0; v < MI; ++v)
                                out[t][v] = __builtin_fmaf(b16, sum[v], __builtin_fmaf(sv, d[v], out[t][v]));
                        }
                    }
                }
            }
        }
    }
};

// An output from its sum in sixteenths: W . x, or silu(G . x) (U . x).
__device__ __forceinline__ float output(float y) { return 16.f * y; }
__device__ __forceinline__ float output(float g, float u) { return 16.f * g / (1.f + expf(-16.f * g)) * (16.f * u); }

// Waves on a SIMD that leave q4_split its registers: a spill would wait for every
// load under way.
constexpr int split_waves(bool f32, int group, int mi, bool two) {
    if (mi == 4) return f32 ? 2 : two ? 3 : 4;
    return two && f32 ? 2 : group == 32 ? 3 : 4;
}

// Each wave takes a piece of k of the block's rows (16 * TN; gated, as many gates
// and ups).
template <class T, class ST, int GROUP, int MI, bool GATED, int TN, int W>
__global__ __launch_bounds__(W* kWave, split_waves(T::code == 0, GROUP, MI, GATED || TN > 1)) void q4_split(
    Q4Args a) {
    constexpr int NT = GATED ? 2 * TN : TN;
    constexpr int CS = MI == 4 ? 1 : T::code == 0 || GATED ? 2 : 4;
    using Z = Tiles<T, ST, GROUP, MI, NT, CS>;
    using S = typename T::store_t;
    constexpr int VT = Z::VT, OCT = Z::OCT;
    constexpr int XL = VT * OCT / kWave;  // octets a lane stages
    // The staged activations, then (after a barrier) the sums to join.
    constexpr int XBYTES = W * sizeof(typename Z::Stage), JBYTES = W * NT * VT * 17 * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[XBYTES > JBYTES ? XBYTES : JBYTES];
    const auto join = reinterpret_cast<float(*)[NT][VT][17]>(lds);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    typename Z::Stage& xs = reinterpret_cast<typename Z::Stage*>(lds)[wave];
    const uint32_t n0 = blockIdx.x * (16 * TN);
    const Rows rows = block_rows<S, VT, 16 * TN, W * kWave>(a, n0);
    if (rows.cnt == 0) return;
    const uint32_t cnt = rows.cnt;
    const uint32_t steps = (a.k + QStep - 1) / QStep;
    const uint32_t st0 = steps * wave / W, st1 = steps * (wave + 1) / W;
    const uint32_t ldx = (uint32_t)a.ldx;  // below 2^25: offsets in a tile fit 32 bits
    const char* const x = reinterpret_cast<const char*>(
        static_cast<const S*>(a.x) + (int64_t)(a.mode == Q4_IDS ? rows.row0 / a.x_div : rows.row0) * a.ldx);

    Z z;
    uint32_t first[NT], end[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t jt = n0 + t % TN * 16;
        first[t] = (jt < a.n ? jt : a.n - 1) + t / TN * a.n;
        end[t] = (1 + t / TN) * a.n;
    }
    z.init(a, (uint64_t)rows.expert * (GATED ? 2 * a.n : a.n), first, end, lane, cnt);
    if (Z::MASKED) {
        for (int o = lane; o < OCT; o += kWave)
#pragma unroll
            for (int p = 0; p < Z::PARTS; ++p) xs.x[p][Z::ROWS - 1][o] = u32x4{0, 0, 0, 0};
    }

    struct Chunk {
        u32x4 x[XL][Z::XR];
        typename Z::Codes q;
    };
    const auto load = [&](Chunk& h, uint32_t s0) {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            if (i * kWave / OCT >= cnt) break;
            const uint32_t v = (i * kWave + lane) / OCT, o = (i * kWave + lane) % OCT;
            z.load_x(h.x[i], x, v < cnt ? v : cnt - 1, ldx, s0, o);
        }
        z.load(h.q, s0, st1);
    };
    const auto step = [&](Chunk& cur, Chunk& nxt, uint32_t s0) {
        if (MI == 1 && s0 + CS < st1) load(nxt, s0 + CS);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            if (i * kWave / OCT >= cnt) break;
            const uint32_t v = (i * kWave + lane) / OCT, o = (i * kWave + lane) % OCT;
            if (v < cnt) z.stage(xs, cur.x[i], v, s0, o);
        }
        // With 16 tokens, only after x has left its registers: there are few.
        if (MI > 1 && s0 + CS < st1) load(nxt, s0 + CS);
        // One wave writes and reads its LDS in order: only the compiler needs telling.
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        z.compute(cur.q, xs, s0, st1);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    Chunk even, odd;
    if (st0 < st1) load(even, st0);
    for (uint32_t s0 = st0; s0 < st1; s0 += 2 * CS) {
        step(even, odd, s0);
        if (s0 + CS < st1) step(odd, even, s0 + CS);
    }

    // Join the W pieces of k.
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < MI; ++v) join[wave][t][MI == 1 ? z.c : 4 * z.c + v][lane & 15] = z.out[t][v];
    __syncthreads();
    S* const y = static_cast<S*>(a.y) + (int64_t)rows.row0 * a.ldy;
    for (uint32_t q = threadIdx.x; q < VT * 16 * TN; q += W * kWave) {
        const uint32_t v = q / (16 * TN), t = q / 16 % TN, j = q % 16, col = n0 + t * 16 + j;
        if (v >= cnt || col >= a.n) continue;
        float sum[2];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            sum[h] = join[0][h * TN + t][v][j];
#pragma unroll
            for (int w = 1; w < W; ++w) sum[h] += join[w][h * TN + t][v][j];
        }
        y[(int64_t)v * a.ldy + col] = narrow(T{}, GATED ? output(sum[0], sum[1]) : output(sum[0]));
    }
}

// Each wave takes 16 * NT rows of W (half gates, half ups) and all of k, for 16 tokens.
template <class T, class ST, int GROUP, bool GATED, int NT, int CS, int W>
__global__ __launch_bounds__(W* kWave, T::code == 0 || GROUP == 32 ? 3 : 4) void q4_block(Q4Args a) {
    using Z = Tiles<T, ST, GROUP, 4, NT, CS>;
    using S = typename T::store_t;
    constexpr int VT = Z::VT, OCT = Z::OCT;
    constexpr int TN = GATED ? NT / 2 : NT, COLS = 16 * TN * W;
    static_assert(VT * OCT % (W * kWave) == 0, "whole octets a lane");
    constexpr int XL = VT * OCT / (W * kWave);
    __shared__ typename Z::Stage xs[2];

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t n0 = blockIdx.x * COLS;
    const Rows rows = block_rows<S, VT, COLS, W * kWave>(a, n0);
    if (rows.cnt == 0) return;
    const uint32_t cnt = rows.cnt;
    const uint32_t steps = (a.k + QStep - 1) / QStep;
    const uint32_t ldx = (uint32_t)a.ldx;  // below 2^25: offsets in a tile fit 32 bits
    const char* const x = reinterpret_cast<const char*>(static_cast<const S*>(a.x) + (int64_t)rows.row0 * a.ldx);

    Z z;
    const uint32_t nw = n0 + wave * (COLS / W);
    uint32_t j[NT], end[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t jt = nw + t % TN * 16;
        j[t] = (jt < a.n ? jt : a.n - 1) + t / TN * a.n;
        end[t] = (1 + t / TN) * a.n;
    }
    z.init(a, (uint64_t)rows.expert * (GATED ? 2 * a.n : a.n), j, end, lane, cnt);

    u32x4 xr[XL][Z::XR];
    const auto load_x = [&](uint32_t s0) {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const uint32_t q = i * (W * kWave) + threadIdx.x, v = q / OCT;
            if (v < cnt) z.load_x(xr[i], x, v, ldx, s0, q % OCT);
        }
    };
    const auto step = [&](typename Z::Codes& cur, typename Z::Codes& nxt, typename Z::Stage& buf, uint32_t s0) {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const uint32_t q = i * (W * kWave) + threadIdx.x, v = q / OCT;
            if (v < cnt) z.stage(buf, xr[i], v, s0, q % OCT);
        }
        if (s0 + CS < steps) {
            load_x(s0 + CS);
            z.load(nxt, s0 + CS, steps);
        }
        // A buffer is written again two chunks later, past the next barrier.
        __syncthreads();
        z.compute(cur, buf, s0, steps);
    };
    typename Z::Codes even, odd;
    load_x(0);
    z.load(even, 0, steps);
    for (uint32_t s0 = 0; s0 < steps; s0 += 2 * CS) {
        step(even, odd, xs[0], s0);
        if (s0 + CS < steps) step(odd, even, xs[1], s0 + CS);
    }

    S* const y = static_cast<S*>(a.y) + (int64_t)rows.row0 * a.ldy;
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const uint32_t col = nw + t * 16 + (lane & 15);
        if (col >= a.n) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (4 * z.c + v < (int)cnt)
                y[(int64_t)(4 * z.c + v) * a.ldy + col] =
                    narrow(T{}, GATED ? output(z.out[t][v], z.out[NT - TN + t][v]) : output(z.out[t][v]));
    }
}

// The instances: up to 4 tokens a tile; 16 tokens with k split over eight waves
// (few blocks), or with the rows split over them.
enum Form { NARROW, SPLIT, SPLIT2, BLOCK };
constexpr int kBlockWaves = 4, kBlockTiles = 2, kBlockSteps = 2;
template <class T, class ST, int GROUP, bool GATED>
const void* pick(Form f) {
    switch (f) {
        case NARROW: return (const void*)&q4_split<T, ST, GROUP, 1, GATED, 1, 4>;
        case SPLIT: return (const void*)&q4_split<T, ST, GROUP, 4, GATED, 1, GATED ? 4 : 8>;
        case SPLIT2:
            if constexpr (!GATED && T::code != 0) return (const void*)&q4_split<T, ST, GROUP, 4, false, 2, 4>;
            return nullptr;
        default: return (const void*)&q4_block<T, ST, GROUP, GATED, kBlockTiles, kBlockSteps, kBlockWaves>;
    }
}
template <class T, class ST>
const void* pick(const Q4Args& a, Form f) {
    switch (a.group) {
        case 32: return a.gated ? pick<T, ST, 32, true>(f) : pick<T, ST, 32, false>(f);
        case 64: return a.gated ? pick<T, ST, 64, true>(f) : pick<T, ST, 64, false>(f);
        default: return a.gated ? pick<T, ST, 128, true>(f) : pick<T, ST, 128, false>(f);
    }
}
template <class T>
const void* pick(const Q4Args& a, Form f) {
    return a.scale_dtype == 1 ? pick<T, TF16>(a, f) : pick<T, TBF16>(a, f);
}

}  // namespace

hipError_t launch_q4(const Q4Args& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_Q4;
    // Sorted: every expert with rows may end inside a tile, and so may the rows
    // without one (the tile added below).
    const uint64_t ends = a.mode == Q4_SORTED ? (a.rows < a.n_experts ? a.rows : a.n_experts) : 0;
    const auto tiles_of = [&](uint32_t vt) { return a.mode == Q4_SORTED ? a.rows / vt + ends : (a.rows + vt - 1ull) / vt; };
    // The sharing form from two blocks a CU on (64 tokens, n = 4096, 8192, 11008: it takes 27, 28,
    // 43 us, the split 16, 29, 40), where rows repeat a staged x and an unpacked code
    // enough: sorted from 1 row an expert on (f16 2048 x 1408, 64 experts: 17.0 us
    // against 19.4 with tiles of 4; f32 23.8 and 26.5), gated 16-bit ones from 3
    // (51.6 and 51.8; at 2 46.1 and 42.5).
    const uint32_t block_cols = 16 * (a.gated ? kBlockTiles / 2 : kBlockTiles) * kBlockWaves;
    const uint32_t per_expert = a.mode == Q4_DENSE ? 5 : a.gated && a.dtype != 0 ? 3 : 1;
    const bool block = a.mode != Q4_IDS && a.rows >= (uint64_t)per_expert * a.n_experts &&
                       tiles_of(16) * ((a.n + block_cols - 1) / block_cols) >= 512;
    // Otherwise 16 tokens a tile from 5 on (11008 x 4096: 3 tokens 9.8 us with tiles
    // of 4, 13.4 with 16; 5 13.5 and 13.9; 8 14.5 and 13.5).
    const bool wide = block || (a.mode != Q4_IDS && a.rows > 4ull * a.n_experts);
    const uint32_t vt = wide ? 16 : 4;
    const uint64_t tiles = a.mode == Q4_IDS ? a.rows : tiles_of(vt) + (a.mode == Q4_SORTED);
    Form f = NARROW;
    uint32_t cols = 16, waves = 4;
    if (block) {
        f = BLOCK;
        cols = block_cols;
        waves = kBlockWaves;
    } else if (wide) {
        // Two tiles share the staged x from 1024 blocks on (gate and up do always; with
        // f32's three parts their registers do not fit): 688 blocks 15.4 us, with two
        // tiles 16.2; 1024 18.8 and 16.5; 2048 33.5 and 29.5.
        f = tiles * ((a.n + 15) / 16) < 1024 || a.gated || a.dtype == 0 ? SPLIT : SPLIT2;
        cols = f == SPLIT ? 16 : 32;
        waves = f == SPLIT && !a.gated ? 8 : 4;
    }
    L->variant = (int)(vt + 256 * cols);
    const void* fn = a.dtype == 0 ? pick<TF32>(a, f) : a.dtype == 1 ? pick<TF16>(a, f) : pick<TBF16>(a, f);
    Q4Args b = a;
    b.tiles = (uint32_t)tiles;
    const uint32_t gy = (uint32_t)(tiles < 32768 ? tiles : 32768);
    void* args[] = {&b};
    return hipLaunchKernel(fn, dim3((a.n + cols - 1) / cols, gy, (uint32_t)((tiles + gy - 1) / gy)),
                           dim3(waves * kWave), args, 0, s);
}

}  // namespace mmk
