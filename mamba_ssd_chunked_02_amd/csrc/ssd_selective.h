// Shared by the selective scan's kernels: how channels, states and tokens lie on
// the lanes of a wave, the moves between its rows, and which tokens a wave takes.
//
// A wave holds 16 channels, lane 16 q + k the q-th quarter of the N states of
// channel k, NS = ceil(N / 4) padded to a power of two, in registers:
//   - what belongs to a (token, channel) is read and computed once, lane 16 q + k
//     for token q of four, and handed to the other rows by swaps of rows;
//   - B and C belong to a (token, state) and are the same for the 16 channels: a
//     register holds 16 / NS tokens' values of the row's NS states, and an
//     operand takes one of them by a row broadcast, for nothing;
//   - a sum over the states is one over registers and the four rows.
#pragma once

#include "ssd_gated.h"

namespace ssd {

constexpr int kSelChannels = 16;       // of a wave
constexpr int kSelBackChannels = 128;  // of a workgroup of the backward pass
constexpr float kLog2e = 1.44269504088896341f;

// Tokens of a tile, whose B and C are NB registers each.
template <int NS>
struct SelTile {
    static constexpr int TT = NS <= 4 ? 16 : 64 / NS;
    static constexpr int NB = TT * NS / 16;
    static constexpr int Q = TT / 4;  // tokens of a lane
};

// ---------------------------------------------------------------- elements
template <typename T>
struct One;
template <>
struct One<float> {
    typedef float raw;
    __device__ static inline raw load(const float* p) { return *p; }
    __device__ static inline float widen(raw v) { return v; }
};
template <>
struct One<bf16_t> {
    typedef uint32_t raw;
    __device__ static inline raw load(const bf16_t* p) { return *(const uint16_t*)p; }
    __device__ static inline float widen(raw v) { return __builtin_bit_cast(float, v << 16); }
};

// One element of y or of a gradient in either type.
__device__ inline void store_one(void* p, int64_t at, bool f32, float v) {
    if (f32) ((float*)p)[at] = v;
    else ((bf16_t*)p)[at] = (bf16_t)v;
}

// ---------------------------------------------------------------- rows
// The halves of a and b: a = [a.lo, b.lo], b = [a.hi, b.hi].
__device__ inline void swap_halves(float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                    false, false);
    const uint32_t lo = r[0], hi = r[1];
    a = __builtin_bit_cast(float, lo);
    b = __builtin_bit_cast(float, hi);
}
// The rows of a and b: a = [a.0, b.0, a.2, b.2], b = [a.1, b.1, a.3, b.3].
__device__ inline void swap_rows(float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                                    false, false);
    const uint32_t lo = r[0], hi = r[1];
    a = __builtin_bit_cast(float, lo);
    b = __builtin_bit_cast(float, hi);
}
// to[j]: row j of v in every row.
__device__ inline void rows_to_all(float v, float (&to)[4]) {
    to[0] = to[2] = v;
    swap_halves(to[0], to[2]);
    to[1] = to[0];
    to[3] = to[2];
    swap_rows(to[0], to[1]);
    swap_rows(to[2], to[3]);
}
// Row j of the result: the sum of v[j] over the four rows.
__device__ inline float sum_rows(const float (&v)[4]) {
    float a = v[0], c = v[2], b = v[1], d = v[3];
    swap_halves(a, c);
    swap_halves(b, d);
    a += c;
    b += d;
    swap_rows(a, b);
    return a + b;
}
// The sum of v over the four rows, in every row.
__device__ inline float sum_all_rows(float v) {
    float w = v;
    swap_halves(v, w);
    v += w;
    w = v;
    swap_rows(v, w);
    return v + w;
}
// Lane I of its row of v.
template <int I>
__device__ inline float row_lane(float v) {
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}

// f(integral_constant<int, 0>) ... <N - 1>
template <int N, int I = 0, typename F>
__device__ inline void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

// ---------------------------------------------------------------- step sizes
// The step size from its raw value, bias and clamp; NaN stays NaN.
struct StepSize {
    bool on, cut;
    float bias, lo, hi;
    __device__ inline StepSize(const DtAct& a, int c) : on(a.on != 0), lo(a.lo), hi(a.hi) {
        cut = on && !(lo == 0.f && hi == __builtin_inff());
        bias = on && a.bias ? a.bias[c] : 0.f;
    }
    __device__ inline float operator()(float raw) const {
        if (!on) return raw;
        float v = softplus_f(raw + bias);
        if (cut) v = v < lo ? lo : v > hi ? hi : v;
        return v;
    }
    // d step / d raw: 0 where the clamp cuts.
    __device__ inline float slope(float raw, float step) const {
        if (!on) return 1.f;
        const float s = sigmoid_f(raw + bias);
        return cut && (step <= lo || step >= hi) ? 0.f : s;
    }
};

}  // namespace ssd
