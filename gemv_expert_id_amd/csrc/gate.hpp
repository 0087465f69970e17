// The gates of the feed-forward products: act(a) = a * sigmoid(z(a)) with
// z = a (SiLU) or z = 2 sqrt(2 / pi) (a + 0.044715 a^3) (GELU, tanh form), and
// act'(a) = s + a s (1 - s) z'(a). All in f32, from f32 pre-activations.
#pragma once

#include "common.hpp"

namespace mmk {

enum Gate { GATE_NONE = 0, GATE_SILU = 1, GATE_GELU = 2 };

constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.044715f;

// sigmoid(z(a)), sigmoid(-z(a)) and z'(a). Both sigmoids come from exp(-|z|), so
// neither loses its small values to a subtraction from 1. Past |a| = 64 they are 0
// or 1 in f32, so the cubic's argument is held there: its powers cannot overflow
// into inf * 0.
struct GateParts {
    float s, rest, slope;
};
__device__ __forceinline__ GateParts gate_parts(int gate, float a) {
    float z = a, dz = 1.f;
    if (gate == GATE_GELU) {
        const float c = __builtin_fminf(__builtin_fmaxf(a, -64.f), 64.f);
        const float c2 = c * c;
        z = kGelu * __builtin_fmaf(kGelu3 * c2, c, c);
        dz = kGelu * __builtin_fmaf(3.f * kGelu3, c2, 1.f);
    }
    const float e = expf(-__builtin_fabsf(z));
    const float big = 1.f / (1.f + e), small = e * big;
    return z >= 0.f ? GateParts{big, small, dz} : GateParts{small, big, dz};
}

__device__ __forceinline__ float gate_act(int gate, float a) { return a * gate_parts(gate, a).s; }

// Gradients of act(g) * u to g and u, times dh.
__device__ __forceinline__ void gate_grad(int gate, float g, float u, float dh, float* dg, float* du) {
    const GateParts p = gate_parts(gate, g);
    *du = dh * (g * p.s);
    *dg = dh * u * __builtin_fmaf(g * p.s * p.rest, p.slope, p.s);
}

}  // namespace mmk
