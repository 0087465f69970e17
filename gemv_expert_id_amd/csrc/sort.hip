// Routed rows in expert order, and back to tokens: the stable sort and its row
// copies, the weighted combination, and the gradients.
//
// The place of a routed row is a count over all ids: the rows of lower experts,
// and those of its own before it. Few rows (sort_small): every token's block
// counts for its own slots while its row of x is under way, one launch and
// nothing exchanged between blocks. Many (sort_plan, then sort_copy): block b
// counts the keys below expert b, which is where its rows begin, then ranks its
// rows in a second pass. Neither needs scratch or atomics on memory; the ids
// are 4 bytes against a row, so reading them more than once is cheap.
//
// The rows are bound by memory: a block takes one token, so a token's row is
// read or written once (in the copy once for each 64 slots), and up to eight
// expert rows are under way at a time. Rows are only element-aligned where pitch or width is odd; the
// hardware takes 16-byte accesses at such addresses, at about 1.4 times the time
// (4096 x 8 bf16 rows: copy 27 us at 2048 wide, 40 at 2047; combine 35 and 54).
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "sort_rule.hpp"

namespace mmk {

namespace {

constexpr int PThreads = 1024;
constexpr int PWaves = PThreads / kWave;
constexpr int CThreads = 256;
constexpr int CWaves = CThreads / kWave;
constexpr int SThreads = 512;  // of the sort in one launch: its blocks share the count
constexpr int SWaves = SThreads / kWave;

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
__device__ __forceinline__ uint32_t wave_total(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)wave_scan(v), kWave - 1);
}
__device__ __forceinline__ float wave_add(float v) {
    const auto add = [&](float o) { v += o; };
    const auto mov = [&](auto ctrl, auto rows) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
            0, (int)__float_as_uint(v), decltype(ctrl)::value, decltype(rows)::value, 0xF, false));
    };
    using std::integral_constant;
    add(mov(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{}));
    add(mov(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{}));
    add(mov(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{}));
    add(mov(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{}));
    add(mov(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{}));
    add(mov(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{}));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), kWave - 1));
}

// Four neighbouring ids' keys (expert, or E for a row without), `pad` past the end.
struct __attribute__((packed, aligned(4))) Ids4 {
    uint32_t v[4];
};
__device__ __forceinline__ void load_keys(const SortArgs& a, int64_t r, int64_t end, uint32_t pad,
                                          uint32_t (&key)[4]) {
    if (r + 4 <= end) {
        const Ids4 q = *reinterpret_cast<const Ids4*>(a.ids + r);
#pragma unroll
        for (int i = 0; i < 4; ++i) key[i] = q.v[i] < a.n_experts ? q.v[i] : a.n_experts;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t id = r + i < end ? a.ids[r + i] : 0u;
            key[i] = r + i < end ? (id < a.n_experts ? id : a.n_experts) : pad;
        }
    }
}

// Up to kSeen * 4096 routed rows the matches of the first pass stay in a register,
// four bits for each load, and the second pass reads no ids. 32768 rows of 64
// experts: 8.80 us, bound by the ids' round trips (65 blocks of 16 waves).
constexpr int kSeen = 16;
__global__ __launch_bounds__(PThreads) void sort_plan(SortArgs a) {
    __shared__ uint32_t s_less[PWaves], s_eq[PWaves];
    constexpr int U = 4, SPAN = kWave * 4;  // loads under way; ids of a wave's load
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint32_t b = blockIdx.x;  // b == E: rows without an expert
    const int64_t R = (int64_t)a.m * a.top_k;
    // Wave w owns a contiguous piece of the routed rows.
    const int64_t piece = (R + PWaves * SPAN - 1) / (PWaves * SPAN) * SPAN;
    const int64_t r0 = wave * piece, r1 = r0 + piece < R ? r0 + piece : R;
    const bool held = piece <= kSeen * SPAN;
    uint64_t seen = 0;
    uint32_t less = 0, eq = 0;
    const auto match = [&](const uint32_t(&key)[4]) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) bits |= key[i] == b ? 1u << i : 0u;
        return bits;
    };
    for (int64_t r = r0; r < r1; r += U * SPAN) {
        uint32_t key[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) load_keys(a, r + u * SPAN + lane * 4, r1, 0xFFFFFFFFu, key[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) less += key[u][i] < b;
            const uint32_t bits = match(key[u]);
            eq += __popc(bits);
            if (held) seen |= (uint64_t)bits << (4 * ((r - r0) / SPAN + u));
        }
    }
    less = wave_total(less);
    eq = wave_total(eq);
    if (lane == 0) { s_less[wave] = less; s_eq[wave] = eq; }
    __syncthreads();
    uint32_t place = 0;
    for (int w = 0; w < PWaves; ++w) place += s_less[w];
    if (threadIdx.x == 0) a.offsets_w[b] = place;
    for (int w = 0; w < wave; ++w) place += s_eq[w];
    if (eq == 0) return;
    // The rows of this expert in one load's ids, `bits` of them each lane's.
    const auto put_places = [&](int64_t r, uint32_t bits) {
        const uint32_t n = __popc(bits), upto = wave_scan(n);
        uint32_t at = place + upto - n;
        for (; bits; bits &= bits - 1, ++at) {
            const uint32_t row = (uint32_t)(r + lane * 4 + __ffs(bits) - 1);
            a.order_w[at] = row;
            a.position_w[row] = at;
        }
        place += (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
    };
    if (held) {
        for (int64_t r = r0; r < r1; r += SPAN, seen >>= 4) put_places(r, (uint32_t)seen & 15u);
        return;
    }
    for (int64_t r = r0; r < r1; r += U * SPAN) {
        uint32_t key[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) load_keys(a, r + u * SPAN + lane * 4, r1, 0xFFFFFFFFu, key[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) put_places(r + u * SPAN, match(key[u]));
    }
}

// 16 bytes of a row that is aligned to its element only. Rows are stored past
// the caches: they are large, and the reads beside them keep their place
// (sort of 512 x 8 f32 rows of 2048 12.8 -> 10.8 us, combination of 8192 x 8
// bf16 rows of 2048 73 -> 67 us, gradient at 2048 x 4 f16 rows of 4096 32 -> 24 us).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
template <class S>
using Chunk = std::conditional_t<sizeof(S) == 4, u32x4_a4, u32x4_a2>;
template <class S, bool NT = false>
__device__ __forceinline__ u32x4 ld_chunk(const S* p) {
    const auto q = reinterpret_cast<const Chunk<S>*>(p);
    if constexpr (NT) return __builtin_nontemporal_load(q);
    else return *q;
}
template <class S>
__device__ __forceinline__ void st_chunk(S* p, u32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<Chunk<S>*>(p));
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

constexpr int KU = kSortSlots;  // slots handled together

// A storage type's bits as they are moved.
template <class T>
using Bits = std::conditional_t<T::code == 0, uint32_t, uint16_t>;

// Elements j .. of a row of `width` at element offset `row`, up to 16 bytes of
// them; zeros, and nothing touched, past the row's end.
template <class S, bool NT = false>
__device__ __forceinline__ u32x4 get(const void* base, int64_t row, uint32_t j, uint32_t width) {
    const S* src = static_cast<const S*>(base) + row + j;
    if (j + 16 / sizeof(S) <= width) return ld_chunk<S, NT>(src);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t q = 0; q < 16 / sizeof(S) - 1; ++q) {
        if (j + q < width) v[q * sizeof(S) / 4] |= (uint32_t)src[q] << (16 * (q & (4 / sizeof(S) - 1)));
    }
    return v;
}
template <class S>
__device__ __forceinline__ void put(void* base, int64_t row, uint32_t j, uint32_t width, u32x4 v) {
    S* dst = static_cast<S*>(base) + row + j;
    if (j + 16 / sizeof(S) <= width) {
        st_chunk(dst, v);
        return;
    }
#pragma unroll
    for (uint32_t q = 0; q < 16 / sizeof(S) - 1; ++q) {
        if (j + q < width) dst[q] = (S)(v[q * sizeof(S) / 4] >> (16 * (q & (4 / sizeof(S) - 1))));
    }
}

// xs[position[t * top_k + s]] = x[t], zeros past the rows that have an expert.
// A block takes a token, one piece of its row and up to kSlots of its slots; the
// rows are moved as bits. Bound by memory: 4096 x 8 bf16 rows of 2048 in 27 us,
// 5.6 TB/s.
constexpr uint32_t kSlots = 64;
template <class S>
__global__ __launch_bounds__(CThreads) void sort_copy(SortArgs a) {
    constexpr int CH = 16 / sizeof(S);
    const uint32_t j = (blockIdx.y * CThreads + threadIdx.x) * CH;
    if (j >= a.width) return;
    const uint32_t live = a.offsets[a.n_experts];
    for (int64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        const u32x4 v = get<S>(a.tokens, t * a.ld_tokens, j, a.width);
        for (uint32_t s0 = blockIdx.z * kSlots; s0 < a.top_k; s0 += gridDim.z * kSlots) {
            const uint32_t s1 = s0 + kSlots < a.top_k ? s0 + kSlots : a.top_k;
            for (uint32_t s = s0; s < s1; ++s) {
                const uint32_t i = a.position[t * a.top_k + s];
                put<S>(a.rows_w, (int64_t)i * a.ld_rows, j, a.width, i < live ? v : u32x4{0, 0, 0, 0});
            }
        }
    }
}

// The whole sort in one launch, for few rows: block 0 counts the offsets, block
// t + 1 the places of token t's slots, KU at a time. 4 x 8 rows of 2048 bf16: 4.6 us, one memory
// round trip and a count; 512 x 8 rows of 2048 f32: 9.8 us, 3.9 TB/s.
template <class S>
__global__ __launch_bounds__(SThreads) void sort_small(SortArgs a) {
    constexpr int CH = 16 / sizeof(S);
    __shared__ uint32_t hist[MM_GROUPED_MAX_E + 1];
    __shared__ uint32_t part[SWaves][KU];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint32_t E = a.n_experts, R = a.m * a.top_k;
    if (blockIdx.x == 0) {
        if (blockIdx.y) return;
        for (uint32_t e = threadIdx.x; e < E; e += SThreads) hist[e] = 0;
        __syncthreads();
        for (uint32_t r = threadIdx.x; r < R; r += SThreads) {
            const uint32_t id = a.ids[r];
            if (id < E) atomicAdd(&hist[id], 1u);
        }
        __syncthreads();
        uint32_t before = 0;
        if (wave == 0) {
            for (uint32_t e0 = 0; e0 < E; e0 += kWave) {
                const uint32_t n = e0 + lane < E ? hist[e0 + lane] : 0;
                const uint32_t upto = wave_scan(n);
                if (e0 + lane < E) a.offsets_w[e0 + lane] = before + upto - n;
                before += (uint32_t)__builtin_amdgcn_readlane((int)upto, kWave - 1);
            }
            if (lane == 0) a.offsets_w[E] = before;
        }
        return;
    }
    const uint32_t t = blockIdx.x - 1;
    const uint32_t j = (blockIdx.y * SThreads + threadIdx.x) * CH;
    u32x4 v = {0, 0, 0, 0};
    if (j < a.width) v = get<S>(a.tokens, (int64_t)t * a.ld_tokens, j, a.width);
    for (uint32_t s0 = 0; s0 < a.top_k; s0 += KU) {
        uint32_t key[KU], n[KU];
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const uint32_t s = s0 + u < a.top_k ? s0 + u : a.top_k - 1;
            const uint32_t id = a.ids[t * a.top_k + s];
            key[u] = id < E ? id : E;
            n[u] = 0;
        }
        for (uint32_t r = threadIdx.x * 4; r < R; r += SThreads * 4) {
            uint32_t k4[4];
            load_keys(a, r, R, 0xFFFFFFFFu, k4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < KU; ++u)
                    n[u] += k4[i] < key[u] + (r + i < t * a.top_k + s0 + u);  // equal ones before it too
        }
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const uint32_t w = wave_total(n[u]);
            if (lane == 0) part[wave][u] = w;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            if (s0 + u >= a.top_k) break;
            uint32_t i = 0;
#pragma unroll
            for (int w = 0; w < SWaves; ++w) i += part[w][u];
            const uint32_t r = t * a.top_k + s0 + u;
            if (threadIdx.x == 0 && blockIdx.y == 0) {
                a.order_w[i] = r;
                a.position_w[r] = i;
            }
            if (j < a.width)
                put<S>(a.rows_w, (int64_t)i * a.ld_rows, j, a.width, key[u] < E ? v : u32x4{0, 0, 0, 0});
        }
        __syncthreads();
    }
}

// Rows that have an expert: all of them without positions.
__device__ __forceinline__ uint32_t live_rows(const SortArgs& a) {
    const uint32_t R = a.m * a.top_k;
    if (!a.position) return R;
    const uint32_t live = a.offsets[a.n_experts];
    return live < R ? live : R;
}

// out[t] = residual[t] + sum_s w[t][s] y[position]; without weights each is 1.
// W: has weights. A block takes one token and one piece of its row. NT: the
// expert rows are read past the caches. Bound by memory: 8192 x 8 bf16 rows of
// 2048 in 61 us, 5.5 TB/s.
template <class T, bool W, bool NT>
__global__ __launch_bounds__(CThreads) void combine(SortArgs a) {
    constexpr int CH = T::Elems16;
    const uint32_t live = live_rows(a);
    const uint32_t j = (blockIdx.y * CThreads + threadIdx.x) * CH;
    if (j >= a.width) return;
    for (int64_t t = blockIdx.x; t < a.m; t += gridDim.x) {
        float acc[CH] = {};
        if (a.residual) unpack<T>(get<Bits<T>>(a.residual, t * a.ld_tokens, j, a.width), acc);
        for (uint32_t s0 = 0; s0 < a.top_k; s0 += KU) {
            u32x4 y[KU];
            bool on[KU];
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const uint32_t r = (uint32_t)t * a.top_k + s0 + u;
                const uint32_t i = s0 + u < a.top_k ? (a.position ? a.position[r] : r) : 0xFFFFFFFFu;
                on[u] = i < live;
                if (on[u]) y[u] = get<Bits<T>, NT>(a.rows, (int64_t)i * a.ld_rows, j, a.width);
            }
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                if (!on[u]) continue;
                const float w = W ? a.weights[(uint32_t)t * a.top_k + s0 + u] : 1.f;
                float f[CH];
                unpack<T>(y[u], f);
#pragma unroll
                for (int q = 0; q < CH; ++q) acc[q] = __builtin_fmaf(w, f[q], acc[q]);
            }
        }
        put<Bits<T>>(a.tokens_w, t * a.ld_tokens, j, a.width, repack<T>(acc));
    }
}

// dy[i] = w dout[t], dw = <dout[t], y[i]>. One wave for each routed row: rows of
// an odd length begin anywhere in 16 bytes, and a wave can take dy's from its
// first 16-byte boundary on, with single elements before and after (2048 x 8
// bf16 rows of 4095: 68 us from the row's start, 62 us so; a block for all
// rows of a token, which reads dout once, 89 us). Bound by memory: 4.6 TB/s there,
// 6.2 TB/s at 2048 x 4 f16 rows of 4096 (24.5 us).
template <class T>
__global__ __launch_bounds__(CThreads) void combine_grad(SortArgs a) {
    using S = typename T::store_t;
    constexpr int CH = T::Elems16, U = 4;  // chunks under way
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t R = a.m * a.top_k, live = live_rows(a);
    for (int64_t r = (int64_t)blockIdx.x * CWaves + threadIdx.x / kWave; r < R;
         r += (int64_t)gridDim.x * CWaves) {
        const uint32_t i = a.position ? a.position[r] : (uint32_t)r;
        const bool on = i < live;
        const float w = on ? a.weights[r] : 0.f;
        float dot = 0.f;
        if (i < R) {
            const S* d = static_cast<const S*>(a.tokens) + (r / a.top_k) * a.ld_tokens;
            const S* y = static_cast<const S*>(a.rows) + (int64_t)i * a.ld_rows;
            S* dy = static_cast<S*>(a.rows_w) + (int64_t)i * a.ld_rows;
            const uint32_t to16 = (uint32_t)(-(uintptr_t)dy & 15) / sizeof(S);
            const uint32_t head = to16 < a.width ? to16 : a.width;
            const uint32_t end = head + (a.width - head) / CH * CH;
            const auto one = [&](uint32_t q) {
                const float g = on ? widen(T{}, d[q]) : 0.f;
                if (on) dot = __builtin_fmaf(g, widen(T{}, y[q]), dot);
                dy[q] = narrow(T{}, on ? w * g : 0.f);
            };
            if (lane < (int)head) one(lane);
            if (end + lane < a.width) one(end + lane);
            for (uint32_t j = head + lane * CH; j < end; j += U * kWave * CH) {
                u32x4 vd[U], vy[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t q = j + u * kWave * CH;
                    if (on && q < end) {
                        vd[u] = ld_chunk(d + q);
                        vy[u] = ld_chunk(y + q);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t q0 = j + u * kWave * CH;
                    if (q0 >= end) break;
                    float g[CH], f[CH], o[CH] = {};
                    if (on) {
                        unpack<T>(vd[u], g);
                        unpack<T>(vy[u], f);
#pragma unroll
                        for (int q = 0; q < CH; ++q) {
                            dot = __builtin_fmaf(g[q], f[q], dot);
                            o[q] = w * g[q];
                        }
                    }
                    st_chunk(dy + q0, repack<T>(o));
                }
            }
        }
        dot = wave_add(dot);
        if (lane == 0) a.dweights_w[r] = on ? dot : 0.f;
    }
}

uint32_t cap(int64_t n) { return (uint32_t)(n < 1 ? 1 : n < (1 << 20) ? n : (1 << 20)); }

}  // namespace

namespace {

// Grid over tokens and pieces of a row (width <= 2^24: at most 2^14 pieces).
dim3 row_grid(int64_t blocks, uint32_t width, int dtype, uint32_t threads) {
    const uint32_t per = threads * (dtype == 0 ? 4 : 8);
    return dim3(cap(blocks), (width + per - 1) / per);
}

}  // namespace

hipError_t launch_sort_plan(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_SORT_PLAN;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel((const void*)&sort_plan, dim3(a.n_experts + 1), dim3(PThreads), args, 0, s);
}

hipError_t launch_sort_rows(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_SORT_ROWS;
    const bool small = sort_launches(a.m, a.top_k) == 1;
    L->variant = small ? 1 : 0;
    const uint32_t threads = small ? SThreads : CThreads;
    const void* fn = small ? (a.dtype == 0 ? (const void*)&sort_small<uint32_t> : (const void*)&sort_small<uint16_t>)
                           : (a.dtype == 0 ? (const void*)&sort_copy<uint32_t> : (const void*)&sort_copy<uint16_t>);
    dim3 grid = row_grid(small ? (int64_t)a.m + 1 : (int64_t)a.m, a.width, a.dtype, threads);
    if (!small) grid.z = a.top_k <= 4096 * kSlots ? (a.top_k + kSlots - 1) / kSlots : 4096;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, s);
}

namespace {

template <class T>
const void* pick_combine(bool w, bool nt) {
    if (!w) return nt ? (const void*)&combine<T, false, true> : (const void*)&combine<T, false, false>;
    return nt ? (const void*)&combine<T, true, true> : (const void*)&combine<T, true, false>;
}

}  // namespace

// From this size on the expert rows pass the caches by. They come from the call
// before: up to about half of the 256 MiB Infinity Cache is still there, more is
// not (268 MB 66.8 -> 62.8 us, 134 MB 35.0 -> 32.1 us; 67 MB 15.5 -> 16.8 us).
constexpr int64_t kPastCacheBytes = 128 << 20;

hipError_t launch_combine(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_COMBINE;
    const bool w = a.weights != nullptr;
    const bool nt = (int64_t)a.m * a.top_k * a.width * (a.dtype == 0 ? 4 : 2) >= kPastCacheBytes;
    const void* fn = a.dtype == 0   ? pick_combine<TF32>(w, nt)
                     : a.dtype == 1 ? pick_combine<TF16>(w, nt)
                                    : pick_combine<TBF16>(w, nt);
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, row_grid(a.m, a.width, a.dtype, CThreads), dim3(CThreads), args, 0, s);
}

hipError_t launch_combine_grad(const SortArgs& a, hipStream_t s, Launched* L) {
    L->kernel = MM_KERNEL_COMBINE_GRAD;
    const void* fn = a.dtype == 0   ? (const void*)&combine_grad<TF32>
                     : a.dtype == 1 ? (const void*)&combine_grad<TF16>
                                    : (const void*)&combine_grad<TBF16>;
    void* args[] = {const_cast<SortArgs*>(&a)};
    return hipLaunchKernel(fn, dim3(cap(((int64_t)a.m * a.top_k + CWaves - 1) / CWaves)), dim3(CThreads),
                           args, 0, s);
}

}  // namespace mmk
