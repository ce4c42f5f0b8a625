// mgs_activation.hpp — the activations of a gated feed-forward layer (internal).
//
// act(g) = g sigmoid(t(g)) with t(g) = g (c1 + c3 g^2): silu has t = g, gelu in
// its form with a hyperbolic tangent t = 2 sqrt(2 / pi) (g + 0.044715 g^3), since
// (1 + tanh z) / 2 = sigmoid(2 z). One set of instructions serves both.
#pragma once

#include <hip/hip_runtime.h>

#include "mgs.h"

namespace mgs {

struct GatedGrad {
    float dg, du, h;
};

struct Activation {
    float c1, c3;
    float e1, e3;            // c1 and c3 times -log2(e)

    // Past 2^13 either way t is so far from zero that the sigmoid is 0 or 1; g^2
    // stays finite. NaN goes on through the products with g.
    static constexpr float kFar = 8192.0f;

#ifdef __HIP_DEVICE_COMPILE__
    // exp2's argument takes four roundings in gelu (the coefficients, g^2, the fma, the
    // product) and two in silu, each 2^-24 of it: e^-t is off by (4 |t| + 2) 2^-24 of
    // itself, silu's by (2 |t| + 2) 2^-24, the sigmoid s by 1 - s of that and four more
    // 2^-24 of the sum and the reciprocal. That is far below a bf16's half step of 2^-8.
    // From t = -87 on, where s is below the normal numbers, it may be zero, also where
    // g s u would be a normal number again.
    __device__ __forceinline__ float sigmoid(float g, float g2) const {
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * fmaf(e3, g2, e1)));
    }
    __device__ __forceinline__ float of(float g) const {
        const float n = __builtin_amdgcn_fmed3f(g, -kFar, kFar);
        return g * sigmoid(n, n * n);
    }
    // h = act(g) u and, from dh, du = dh act(g) and
    // dg = dh u act'(g), act'(g) = s + act(g) (1 - s) t'(g).
    __device__ __forceinline__ GatedGrad grad(float dh, float g, float u) const {
        const float n = __builtin_amdgcn_fmed3f(g, -kFar, kFar), n2 = n * n;
        const float s = sigmoid(n, n2), a = g * s;
        const float slope = fmaf(a * (1.0f - s), fmaf(3.0f * c3, n2, c1), s);
        return {dh * u * slope, dh * a, a * u};
    }
#else
    // (the host pass only parses the kernels)
    __device__ float of(float g) const { return g; }
    __device__ GatedGrad grad(float dh, float g, float u) const { return {dh, g, u}; }
#endif
};

// Of MGS_ACT_SILU or MGS_ACT_GELU.
inline Activation activation(int act) {
    const double c1 = act == MGS_ACT_GELU ? 1.5957691216057308 : 1.0, c3 = act == MGS_ACT_GELU ? c1 * 0.044715 : 0.0;
    const double log2e = 1.4426950408889634;
    return {(float)c1, (float)c3, (float)(-c1 * log2e), (float)(-c3 * log2e)};
}

}  // namespace mgs
