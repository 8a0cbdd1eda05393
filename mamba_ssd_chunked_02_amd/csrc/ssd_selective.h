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

constexpr int kSelChannels = 16;  // of a wave
constexpr int kSelBackWaves = 4;  // of a workgroup of the backward pass
constexpr int kSelBackChannels = kSelBackWaves * kSelChannels;
constexpr float kLog2e = 1.44269504088896341f;

// Tokens of a tile, whose B and C are NB registers each.
template <int STATES>
struct SelTile {
    static constexpr int NS = STATES;
    static constexpr int TT = NS == 1 ? 16 : NS <= 8 ? 8 : 4;
    static constexpr int NB = TT * NS / 16;
    static constexpr int Q = TT / 4;  // tokens of a lane
};

// The same for the backward pass, which holds a tile's states and decays in
// registers; SUB tokens lie between two states kept in LDS.
template <int STATES>
struct SelBack {
    static constexpr int NS = STATES;
    static constexpr int TT = NS == 1 ? 16 : NS <= 4 ? 8 : 4;
    static constexpr int NB = TT * NS / 16;
    static constexpr int Q = TT / 4;
    static constexpr int SUB = NS <= 4 ? TT : 16;
};

// f(integral_constant<int, 0>) ... <N - 1>
template <int N, int I = 0, typename F>
__device__ inline void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

// ---------------------------------------------------------------- elements
// One element as it is loaded from a buffer, 0 where the offset lies behind its end.
constexpr int kSelBufferWord3 = 0x00020000;            // gfx9 untyped data
constexpr uint32_t kSelNowhere = 0x80000000u;          // behind the end of any of the buffers here
template <typename T>
struct One;
template <>
struct One<float> {
    typedef float raw;
    __device__ static inline raw load(const float* p) { return *p; }
    __device__ static inline raw load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        const uint32_t v = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
        return __builtin_bit_cast(float, v);
    }
    __device__ static inline void store(__amdgpu_buffer_rsrc_t r, uint32_t at, float v) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, at, 0, 0);
    }
    __device__ static inline float widen(raw v) { return v; }
};
template <>
struct One<bf16_t> {
    typedef uint32_t raw;
    __device__ static inline raw load(const bf16_t* p) { return *(const uint16_t*)p; }
    __device__ static inline raw load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
    }
    __device__ static inline void store(__amdgpu_buffer_rsrc_t r, uint32_t at, float v) {
        const bf16_t n = (bf16_t)v;
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, n), r, at, 0, 0);
    }
    __device__ static inline float widen(raw v) { return __builtin_bit_cast(float, v << 16); }
};

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
// Row j of the result: the sum of v[j] over the four rows.  A swap takes a register
// two wait states after a vector instruction wrote it, which the compiler sees to for
// its own instructions, but not for dot_row's, whose results come here: hence the wait.
__device__ inline float sum_rows(const float (&v)[4]) {
    float a = v[0], c = v[2], b = v[1], d = v[3];
    asm("s_nop 1" : "+v"(a), "+v"(b), "+v"(c), "+v"(d));
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

// What the wave wrote to LDS before this is read after it: LDS works for a wave in
// order, the compiler has to as well.
__device__ inline void in_wave_order() {
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// acc = (FIRST) or acc += src[lane F + j of its row] v[j] for j = 0..3: the
// multiplication takes its operand across the row, which the compiler does only for
// plain products (with a move otherwise: 7 cycles in place of 4.6).  The operand must
// not have been written in the two instructions before; nor may another lane take a
// result in the two behind (sum_rows waits).
template <int F, bool FIRST>
__device__ inline void dot_row4(float& acc, float src, float v0, float v1, float v2, float v3) {
    if constexpr (FIRST)
        asm("s_nop 1\n\t"
            "v_mul_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
            : "=&v"(acc)
            : "v"(src), "v"(v0), "v"(v1), "v"(v2), "v"(v3), "n"(F), "n"(F + 1), "n"(F + 2), "n"(F + 3));
    else
        asm("s_nop 1\n\t"
            "v_fmac_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
            : "+v"(acc)
            : "v"(src), "v"(v0), "v"(v1), "v"(v2), "v"(v3), "n"(F), "n"(F + 1), "n"(F + 2), "n"(F + 3));
}
// acc_j += src[lane F + j of its row] v; the results as dot_row4's.
template <int F>
__device__ inline void add_row4(float& a0, float& a1, float& a2, float& a3, float src, float v) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %4, %5 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %5 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %5 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "+v"(a0), "+v"(a1), "+v"(a2), "+v"(a3)
        : "v"(src), "v"(v), "n"(F), "n"(F + 1), "n"(F + 2), "n"(F + 3));
}
// The same for the NS states of a token, whose first one is at lane F; the dot
// product is returned.
template <int F, int NS>
__device__ inline float dot_row(float src, const float (&v)[NS]) {
    float acc = 0.f;
    if constexpr (NS >= 4) {
        unroll<NS / 4>([&](auto four) {
            constexpr int o = 4 * decltype(four)::value;
            dot_row4<F + o, o == 0>(acc, src, v[o], v[o + 1], v[o + 2], v[o + 3]);
        });
    } else {
        unroll<NS>([&](auto one) {
            constexpr int j = decltype(one)::value;
            acc = __builtin_fmaf(row_lane<F + j>(src), v[j], acc);
        });
    }
    return acc;
}
template <int F, int NS>
__device__ inline void add_row(float (&acc)[NS], float src, float v) {
    if constexpr (NS >= 4) {
        unroll<NS / 4>([&](auto four) {
            constexpr int o = 4 * decltype(four)::value;
            add_row4<F + o>(acc[o], acc[o + 1], acc[o + 2], acc[o + 3], src, v);
        });
    } else {
        unroll<NS>([&](auto one) {
            constexpr int j = decltype(one)::value;
            acc[j] = __builtin_fmaf(row_lane<F + j>(src), v, acc[j]);
        });
    }
}

// ---------------------------------------------------------------- rows in memory
// The compiler shall keep one scalar pointer a tensor, not one for every load of a
// tile (which runs out of scalar registers and then adds in vector ones).
__device__ inline const char* opaque(const char* p) {
    asm volatile("" : "+s"(p));
    return p;
}
// A tensor's rows of a tile as a buffer that ends with the last row that is there:
// rows behind it read as 0 and are not written.
struct TileRows {
    __amdgpu_buffer_rsrc_t r;
    uint32_t lane, stride;
    // row: a constant
    __device__ inline uint32_t at(int row) const { return lane + row * stride; }
};
// A tensor of rows as a wave reads it, from the first row of a tile of TT: lane
// 16 q + k takes row 4 i + q of its channel.
template <int TT>
struct RowsOf {
    const char* p;
    uint32_t stride, width, lane;  // bytes
    __device__ inline RowsOf(const void* base, int64_t row, int64_t elements, int size, int C, int c, int q)
        : p((const char*)base + row * elements * size), stride((uint32_t)elements * size), width((uint32_t)C * size),
          lane(q * stride + c * size) {}
    __device__ inline void move(int rows) { p = opaque(p + rows * (int64_t)stride); }
    __device__ inline TileRows tile(int left) const {
        const uint32_t bytes = (min(left, TT) - 1) * stride + width;
        return {__builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, (int)bytes, kSelBufferWord3), lane,
                stride};
    }
};
// B or C of a tile of geometry G: register i holds state f % NS of the row's quarter
// for token f / NS, f = 16 i + k; 0 for states behind the last one.
template <typename T, typename G>
struct StatesOf {
    static constexpr int NS = G::NS, P = 16 / NS;  // tokens of a register
    const char* p;
    uint32_t stride, width, lane;
    __device__ inline StatesOf(const void* base, int64_t row, int64_t elements, int first, int N, int q, int k)
        : p((const char*)base + (row * elements + first) * (int64_t)sizeof(T)), stride((uint32_t)elements * sizeof(T)),
          width(N * sizeof(T)) {
        const int s = q * NS + k % NS;
        lane = s < N ? k / NS * stride + s * (uint32_t)sizeof(T) : kSelNowhere;
    }
    __device__ inline void move(int rows) { p = opaque(p + rows * (int64_t)stride); }
    __device__ inline void load(int left, typename One<T>::raw (&to)[G::NB]) const {
        const uint32_t bytes = (min(left, G::TT) - 1) * stride + width;
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), (short)0, (int)bytes, kSelBufferWord3);
#pragma unroll
        for (int i = 0; i < G::NB; ++i) to[i] = One<T>::load(r, lane + i * P * stride);
    }
    __device__ static inline void widen(const typename One<T>::raw (&r)[G::NB], float (&to)[G::NB]) {
#pragma unroll
        for (int i = 0; i < G::NB; ++i) to[i] = One<T>::widen(r[i]);
    }
};
// y and dy may be of the other type than x.
__device__ inline uint32_t load_either(const TileRows& r, int row, bool f32) {
    return f32 ? __builtin_amdgcn_raw_buffer_load_b32(r.r, r.at(row), 0, 0)
               : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r.r, r.at(row), 0, 0);
}
__device__ inline float widen_either(uint32_t v, bool f32) {
    const uint32_t bits = f32 ? v : v << 16;
    return __builtin_bit_cast(float, bits);
}

// ---------------------------------------------------------------- step sizes
// log2(e) A, the factor of the step size in a decay's exponent.  Kept finite, so
// that a step of 0 leaves the state as it is whatever A is: a tile's rows behind the
// last token take such steps.  NaN stays NaN.
__device__ inline float decay_rate(float A) {
    return __builtin_elementwise_minimum(__builtin_elementwise_maximum(A * kLog2e, -3.4028234e38f), 3.4028234e38f);
}

// softplus(v) = max(v, 0) + log(1 + u), u = exp(-|v|): 14 operations, off by less than 4
// of 2^-24 down to v = -87 (measured on 2^16 values over the range: 2.7 for v >= 0, 3.8
// for v > -15, 2.7 below).  The exponent's product is taken in two parts, with the second
// part of log2(e), without which it would be off by |v| / 4 more (and 0.5% of the packed
// forward's time less); what 1 + u loses of u is added again.  NaN stays NaN; exp(v) too
// small for a normal number counts as 0.
__device__ inline float softplus_quick(float v) {
    const float n = __builtin_elementwise_maximum(-fabsf(v), -88.f), t = n * 0x1.715476p+0f;
    const float lo = __builtin_fmaf(n, 0x1.4ae0cp-26f, __builtin_fmaf(n, 0x1.715476p+0f, -t));
    const float u0 = __builtin_amdgcn_exp2f(t);
    const float u = __builtin_fmaf(u0 * 0x1.62e43p-1f, lo, u0), w = 1.f + u;
    return __builtin_elementwise_maximum(v, 0.f) +
           __builtin_fmaf(__builtin_amdgcn_logf(w), 0x1.62e43p-1f, u - (w - 1.f));
}

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
        const float v = softplus_quick(raw + bias);
        return __builtin_elementwise_minimum(__builtin_elementwise_maximum(v, lo), hi);
    }
    // d step / d raw: 0 where the clamp cuts.
    __device__ inline float slope(float raw, float step) const {
        if (!on) return 1.f;
        const float s = sigmoid_f(raw + bias);
        return cut && (step <= lo || step >= hi) ? 0.f : s;
    }
};

// ---------------------------------------------------------------- states that are not there
// A lane's states behind the last one are 0, as their B and C are, and so add nothing to a
// sum over states -- but for 0 times an infinity, a NaN that would stay.  A tile with such
// a factor is computed with the masks, which put these states back to 0: forward once
// more, when the NaN has shown, backward in place of the plain way.
__device__ inline bool finite(float v) { return fabsf(v) < __builtin_inff(); }
template <int NS>
struct There {
    uint32_t m[NS];
    __device__ inline There(int N, int q) {
        asm volatile("" : "+s"(N));  // here, not in front of the loop over tiles, where nobody needs them
#pragma unroll
        for (int j = 0; j < NS; ++j) m[j] = q * NS + j < N ? 0xffffffffu : 0u;
    }
    __device__ inline float operator()(int j, float v) const {
        return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & m[j]);
    }
};
struct Everywhere {
    __device__ inline Everywhere(int, int) {}
    __device__ inline float operator()(int, float v) const { return v; }
};

// ---------------------------------------------------------------- items
__device__ inline int64_t uniform64(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
// An item is the same for all lanes: in scalar registers.
__device__ inline SelItem uniform_item(SelItem e) {
    e.seq = uniform64(e.seq);
    e.lo = uniform64(e.lo);
    e.n = uniform64(e.n);
    e.first = uniform64(e.first);
    e.index = uniform64(e.index);
    e.last = __builtin_amdgcn_readfirstlane(e.last);
    return e;
}

// ---------------------------------------------------------------- carry
// Along the items of a sequence, in place: what an item ends with from zero becomes
// what it ends with, h that in front of the first one.  p and steps: the first item's,
// dp and ds from one item to the next.  Items' values are read some ahead of the
// chain, whose latency this is.
__device__ inline void carry(float* p, int64_t dp, const float* steps, int64_t ds, int64_t items, float A, float h) {
    constexpr int AHEAD = 16;
    for (int64_t i = 0; i < items; i += AHEAD, p += AHEAD * dp, steps += AHEAD * ds) {
        const int n = (int)min(items - i, (int64_t)AHEAD);
        float v[AHEAD], a[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int o = min(j, n - 1);
            v[j] = p[o * dp];
            a[j] = steps[o * ds];
        }
        const float in = h;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (j >= n) break;
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * a[j]), h, v[j]);
            p[j * dp] = h;
        }
        // An item's factor may underflow or overflow where no token's does, but is a positive
        // number: 0 and infinity pass it as they are.  Looked into where a NaN came of it.
        if (h == h) continue;
        h = in;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (j >= n) break;
            const float e = A * a[j];
            const bool kept = (h == 0.f || fabsf(h) == __builtin_inff()) && fabsf(e) < __builtin_inff();
            h = kept ? h + v[j] : __builtin_fmaf(__builtin_amdgcn_exp2f(e), h, v[j]);
            p[j * dp] = h;
        }
    }
}

}  // namespace ssd
