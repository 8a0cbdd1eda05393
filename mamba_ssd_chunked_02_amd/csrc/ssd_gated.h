// Shared by the gated recurrence's kernels and the conv1d gradients: four
// channels as they are loaded, and the gates of one element.
#pragma once

#include "ssd_device.h"
#include "ssd_rows.h"

namespace ssd {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------- four channels as loaded
// bf16 channels stay in the two words they were loaded as (a vector of 16-bit
// elements that meets a branch takes a register for every element).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    typedef f32x4 type;
    __device__ static inline f32x4 widen(f32x4 v) { return v; }
    __device__ static inline f32x4 all(float v) { return f32x4{v, v, v, v}; }
};
template <>
struct Raw<bf16_t> {
    typedef uint32_t type __attribute__((ext_vector_type(2)));
    __device__ static inline f32x4 widen(type v) {
        return f32x4{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xffff0000u),
                     __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xffff0000u)};
    }
    // v exact in bf16
    __device__ static inline type all(float v) {
        const uint32_t h = __builtin_bit_cast(uint32_t, v), w = h | h >> 16;
        return type{w, w};
    }
};

// ---------------------------------------------------------------- gates
// sigmoid with the hardware exponential and reciprocal (1 ulp each).
__device__ inline float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

// softplus(v) = max(v, 0) + log(1 + u), u = exp(-|v|) <= 1, to about 4 of 2^-24.
// u: the product with log2(e) in two parts, the small one to first order;
// log(1 + u) = 2 atanh(s), s = u / (2 + u) <= 1/3: the series to s^13 (the first
// term left out is below 2^-25 of it).  Below -87, where u is no normal number, 0.
// 25 operations; expf and log1pf take four
// times as many, which the single-token step would wait for.
__device__ inline float softplus_f(float v) {
    const float n0 = -fabsf(v), n = n0 < -88.f ? -88.f : n0, t = n * 0x1.715476p+0f;  // NaN stays
    const float lo = __builtin_fmaf(n, 0x1.715476p+0f, -t) + n * 0x1.4ae0cp-26f;
    const float u0 = __builtin_amdgcn_exp2f(t), u = __builtin_fmaf(u0, lo * 0x1.62e43p-1f, u0);
    const float s = u * __builtin_amdgcn_rcpf(2.f + u), q = s * s;
    float p = 2.f / 13.f;
    p = __builtin_fmaf(p, q, 2.f / 11.f);
    p = __builtin_fmaf(p, q, 2.f / 9.f);
    p = __builtin_fmaf(p, q, 2.f / 7.f);
    p = __builtin_fmaf(p, q, 2.f / 5.f);
    p = __builtin_fmaf(p, q, 2.f / 3.f);
    p = __builtin_fmaf(p, q, 2.f);
    return v < -87.f ? 0.f : fmaxf(v, 0.f) + s * p;
}

// The factor of sigmoid(r) in log a: -rate softplus(lam).  However large it is, a
// gate that is nearly closed makes a decay of it that counts, so nothing may be
// cut off before the gate has multiplied it but what keeps it finite (a gate of 0
// times infinity is no number): no lower than -1e30.  NaN stays NaN.
__device__ inline float decay_factor(float lam, float rate) {
    const float k = -rate * softplus_f(lam);
    return k < -1e30f ? -1e30f : k;
}

// exp(v) - 1 for v in [-0.35, 0]: v times the minimax polynomial of degree 4 of
// (exp(v) - 1) / v there, fitted by exchange on its relative error (0.22 of
// 2^-24); 2 of 2^-24 with the roundings.
constexpr float kSlowDecay = -0.35f;
__device__ inline float expm1_slow(float v) {
    float p = 0x1.d82f32p-8f;
    p = __builtin_fmaf(p, v, 0x1.528df0p-5f);
    p = __builtin_fmaf(p, v, 0x1.553f22p-3f);
    p = __builtin_fmaf(p, v, 0x1.ffff82p-2f);
    p = __builtin_fmaf(p, v, 1.f);
    return p * v;
}

// a = exp(v) and m = 1 - a^2 = -e (1 + a), e = a - 1, with no cancellation
// however near a is to 1, and w, which holds both: e (<= 0) where v >= -0.35,
// elsewhere a itself, no less than kLeastDecay (> 0), which is taken off again where
// w is read: a gradient multiplies an a that underflowed by the decay factor, which
// may be 1e30, and has to find 0.  slow (the same for a wave): no channel of the wave
// decays by more than 0.35 a token, so that no element takes the exponential.
constexpr float kLeastDecay = 1e-37f;

// a of one held decay; what is taken off is below half a step of any a over 2e-30.
__device__ inline float held_decay(float held) { return held + (held > 0.f ? -kLeastDecay : 1.f); }

struct Decay {
    f32x4 a, m, w;
    __device__ inline void from_log(f32x4 v, bool slow) {
        if (slow) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = expm1_slow(v[c]);
                a[c] = 1.f + w[c];
                m[c] = __builtin_fmaf(-w[c], a[c], -w[c]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = expm1_slow(v[c]),
                            q = fmaxf(__builtin_amdgcn_exp2f(v[c] * 1.44269504088896341f), kLeastDecay);
                const bool far = v[c] < kSlowDecay;
                const float e = far ? q - 1.f : p;
                a[c] = far ? q : 1.f + p;
                w[c] = far ? q : p;
                m[c] = __builtin_fmaf(-e, a[c], -e);
            }
        }
    }
    __device__ inline void from_held(f32x4 held, bool slow) {
        if (slow) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[c] = 1.f + held[c];
                m[c] = __builtin_fmaf(-held[c], a[c], -held[c]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float e = held[c] > 0.f ? held[c] - 1.f : held[c];
                a[c] = held_decay(held[c]);
                m[c] = __builtin_fmaf(-e, a[c], -e);
            }
        }
    }
};

// a of a held decay.
__device__ inline f32x4 decay_of(f32x4 held, bool slow) {
    f32x4 a;
    if (slow) {
#pragma unroll
        for (int c = 0; c < 4; ++c) a[c] = 1.f + held[c];
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) a[c] = held_decay(held[c]);
    }
    return a;
}

}  // namespace ssd
