// Gradients of the selective scan on gfx950.  With u = dy silu(z) the gradient of
// what the gate multiplies and a = exp(dt A), from the last token to the first:
//   g = u C + a' g'          (a', g': of the token after; the adjoint of the state)
//   s = sum_n g B,  w_n = (a g)_n h_n of the token before
//   dx = dt s + D u,  d dt = x s + sum_n A w,  dz = dy (sum_n h C + D x) silu'(z)
//   dA = sum_t dt w,  dB = sum_c g dt x,  dC = sum_c u h,  dD = sum_t u x
// and draw = d dt times the slope of the step size, dbias its sum over tokens.
//
// As the forward pass, with the tokens reversed: items' adjoints from zero, their
// carry, then the gradients.  The states are computed again from the saved ones
// (every 64 tokens): first those entering every 8 tokens (16 for less than 5 states or
// more than 16), which a lane keeps in LDS, then a tile's, which it keeps in registers
// with the decays.
//
// The vector ALU bounds it: 33.7 instructions a (token, channel, state) in the gradients'
// kernel for 16 states: 4 for states and decays, 3.5 for the states once more in front of
// that, 9 for the adjoint, the products and their sums over states and tokens, 3 for dB's
// and dC's sums over channels; the rest belongs to a (token, channel) or is the compiler's:
// of 1764 vector instructions in the loop over tiles (two forms of a tile) 207 are moves
// and 89 lane reads of spilled scalars, of 1605 in that over chunks 40 and 168.  It holds
// 208 registers, so two waves a SIMD, and is busy 80% of their cycles.  8 x 2048 x 5120 x
// 16, bf16: 1.62 ms, the adjoints 0.25, the sums 0.06.  Three waves a SIMD spill (2.56
// against 2.0 ms at that time), as do two channels a lane; fp32 matrix products for the
// sums over channels do not run beside the vector ALU.  For 33 to 64 states two waves
// spill as well, 64 to 71 registers of a lane: 0.53 T states a second, where 16 states
// reach 0.70.
#include <algorithm>
#include <type_traits>

#include "ssd_column_sum.h"
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kWaves = kSelBackWaves;  // of a workgroup
constexpr int64_t kMaxBlocks = 1 << 22;
constexpr float kLn2 = 0.693147180559945309f;

// ---------------------------------------------------------------- sums over channels
// Which half of its 16, 8, 4 and 2 lanes a lane is in, as masks: a select by one
// takes 4.5 cycles, one by a condition code in vcc 24.
struct Halves {
    uint32_t m[4];
    __device__ inline Halves(int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = k >> i & 1 ? 0xffffffffu : 0u;
            asm volatile("" : "+v"(m[i]));  // or the compiler makes conditions of them again
        }
    }
};
template <int CTRL>
__device__ inline float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ inline float pick(uint32_t m, float set, float clear) {
    const uint32_t s = __builtin_bit_cast(uint32_t, set), c = __builtin_bit_cast(uint32_t, clear), r = (m & s) | (~m & c);
    return __builtin_bit_cast(float, r);
}
// a and b, each summed over twice as many lanes, in one: a lane keeps the value of
// its half and takes it from the lane opposite.
template <int STEP>
__device__ inline float halve(float a, float b, const Halves& h) {
    // row_mirror, row_half_mirror, quad_perm:[3,2,1,0], quad_perm:[1,0,3,2]
    constexpr int CTRL = STEP == 0 ? 0x140 : STEP == 1 ? 0x141 : STEP == 2 ? 0x1b : 0xb1;
    const uint32_t m = h.m[3 - STEP];
    return pick(m, b, a) + dpp<CTRL>(pick(m, a, b));
}
// Sums over the 16 channels of a row of 16 values, NS states of P = 16 / NS tokens,
// taken as they come: lane P j + t of the row gets the sum for state j of token t.
// The states' halves are joined first, so that a token leaves one value behind.
template <int NS, int STEP, int N>
__device__ inline float join(const float (&v)[N], const Halves& h) {
    if constexpr (N == 1) {
        return v[0];
    } else {
        float to[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) to[i] = halve<STEP>(v[i], v[i + N / 2], h);
        return join<NS, STEP + 1>(to, h);
    }
}
// Both gradients' NS states of a token, each in one value.  For four states the adds
// write only the lanes of their half, 6 operations a value in place of 9; every
// operand is written at least two instructions before its lanes are exchanged.
template <int NS>
__device__ inline void join_states(const float (&v)[NS], const float (&w)[NS], const Halves& h, float& tv, float& tw) {
    if constexpr (NS == 4) {
        float a, b, c, d;
        asm("s_nop 1\n\t"
            "v_add_f32_dpp %2, %6, %6 row_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %2, %8, %8 row_mirror row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %3, %7, %7 row_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %3, %9, %9 row_mirror row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %4, %10, %10 row_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %4, %12, %12 row_mirror row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %5, %11, %11 row_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %5, %13, %13 row_mirror row_mask:0xf bank_mask:0xc\n\t"
            "v_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %0, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
            "v_add_f32_dpp %1, %4, %4 row_half_mirror row_mask:0xf bank_mask:0xf\n\t"
            "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
            "s_nop 1"
            : "=&v"(tv), "=&v"(tw), "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
            : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(w[0]), "v"(w[1]), "v"(w[2]), "v"(w[3]));
    } else {
        tv = join<NS, 0>(v, h);
        tw = join<NS, 0>(w, h);
    }
}
constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }
template <int NS>
__device__ inline float join_tokens(const float (&v)[16 / NS], const Halves& h) {
    return join<NS, log2_of(NS)>(v, h);
}
// The state and the token of lane l of a row.
template <int NS>
__device__ inline int joined_state(int l) {
    return l / (16 / NS);
}
template <int NS>
__device__ inline int joined_token(int l) {
    return l % (16 / NS);
}

// ---------------------------------------------------------------- adjoints of items, from zero
// The gradient that an item hands to the token before it if none enters at its end,
// for all items but a sequence's first.
template <typename T, int NS>
__global__ __launch_bounds__(256, NS <= 4 ? 5 : 3) void selective_adjoint_kernel(SelArgs a, SelLayout lay, float* ends, float* steps) {
    typedef SelTile<NS> G;
    constexpr int TT = G::TT, Q = G::Q;
    // what the rows of a wave hand to each other: step sizes and the output's gradient
    __shared__ float s_x[4][TT][16][2];
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = a.C / a.G, nblk = (per + 4 * kSelChannels - 1) / (4 * kSelChannels) * a.G;
    const int64_t work = lay.places * nblk;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / (nblk / a.G);
        const SelItem e = uniform_item(sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place));
        if (e.seq < 0 || e.index == 0) continue;
        const int c0 = g * per + ((cb - g * (nblk / a.G)) * 4 + wave) * kSelChannels, end = (g + 1) * per;
        if (c0 >= end) continue;
        const bool on = c0 + k < end;
        const int c = on ? c0 + k : end - 1;
        const int n = (int)e.n;
        float A[NS], ga[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int s = q * NS + j;
            A[j] = s < a.N ? decay_rate(a.A[(int64_t)c * a.N + s]) : 0.f;
            ga[j] = 0.f;
        }
        const StepSize step(a.act, c);
        float total = 0.f;
        typedef RowsOf<TT> Rows;
        const int size = (int)sizeof(T);
        Rows dts(a.dt, e.lo, a.dt_stride, size, a.C, c, q), zs(a.z, e.lo, a.z_stride, size, a.C, c, q);
        Rows dys(a.dy, e.lo, a.C, a.y_f32 ? 4 : 2, a.C, c, q);
        StatesOf<T, G> cs(a.Cm, e.lo, a.c_stride, g * a.N, a.N, q, k);
        struct Raw {
            typename One<T>::raw dt[Q], z[Q], c[G::NB];
            uint32_t dy[Q];
        };
        auto move = [&](int rows) {
            dts.move(rows);
            dys.move(rows);
            cs.move(rows);
            if (a.z) zs.move(rows);
        };
        auto load = [&](int left, Raw& r) {
            const TileRows td = dts.tile(left), ty = dys.tile(left), tz = zs.tile(left);
            cs.load(left, r.c);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                r.dt[i] = One<T>::load(td.r, td.at(4 * i));
                r.dy[i] = load_either(ty, 4 * i, a.y_f32);
                if (a.z) r.z[i] = One<T>::load(tz.r, tz.at(4 * i));
            }
            move(-TT);
        };
        // the tile's first `left` tokens; a row behind them takes a step of 0, and its dy is 0
        auto tile = [&](int left, const Raw& r) {
            float cc[G::NB];
            cs.widen(r.c, cc);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                float dt = step(One<T>::widen(r.dt[i]));
                if (left < TT) dt = 4 * i + q < left ? dt : 0.f;
                float u = widen_either(r.dy[i], a.y_f32);
                if (a.z) {
                    const float z = One<T>::widen(r.z[i]);
                    u *= z * sigmoid_f(z);
                }
                total += dt;
                *(f32x2*)s_x[wave][4 * i + q][k] = f32x2{dt, u};
            }
            in_wave_order();
            f32x2 next = *(const f32x2*)s_x[wave][TT - 1][k];
            unroll<TT>([&](auto token) {
                constexpr int t = TT - 1 - decltype(token)::value;
                const f32x2 now = next;
                if (t > 0) next = *(const f32x2*)s_x[wave][t > 0 ? t - 1 : 0][k];
                add_row<t * NS % 16>(ga, cc[t * NS / 16], now[1]);
#pragma unroll
                for (int j = 0; j < NS; ++j) ga[j] *= __builtin_amdgcn_exp2f(now[0] * A[j]);
            });
            in_wave_order();
        };
        Raw cur, nxt;
        int t0 = (n - 1) / TT * TT;
        move(t0);
        load(n - t0, nxt);
        for (; t0 >= 0; t0 -= TT) {
            cur = nxt;
            if (t0) load(TT, nxt);
            tile(n - t0, cur);
        }
        total = sum_all_rows(total);
        if (!on) continue;
#pragma unroll
        for (int j = 0; j < NS; ++j) ends[(place * a.C + c) * (4 * NS) + q * NS + j] = ga[j];
        if (q == 0) steps[place * a.C + c] = total;
    }
}

// Carries the adjoints over the items of a sequence from its end, in place: what
// item j hands to the token before it.
__global__ __launch_bounds__(256) void selective_carry_back_kernel(SelArgs a, SelLayout lay, float* ends,
                                                                   const float* steps, int padded) {
    const int64_t row = (int64_t)a.C * padded, work = (row + 255) / 256;
    for (int64_t w = blockIdx.x; w < work * a.nseq; w += gridDim.x) {
        const int64_t s = w / work, at = (w - s * work) * 256 + threadIdx.x;
        if (at >= row) continue;
        const RowRange r = seq_range(a.cu, a.L, a.T, s);
        const int64_t items = (r.hi - r.lo + lay.item - 1) / lay.item;
        if (items < 2) continue;
        const int c = (int)(at / padded), n = (int)(at - (int64_t)c * padded);
        const bool there = n < a.N;
        const float A = there ? decay_rate(a.A[(int64_t)c * a.N + n]) : 0.f;
        const float h = a.dfinal && there ? a.dfinal[(s * a.C + c) * a.N + n] : 0.f;
        const int64_t place = sel_place(a.cu != nullptr, s, r.lo, a.L, lay.item) + items - 1;
        carry(ends + place * row + at, -row, steps + place * a.C + c, -(int64_t)a.C, items - 1, A, h);
    }
}

// ---------------------------------------------------------------- gradients
template <typename T, int NS>
struct RawBack {
    typedef SelBack<NS> G;
    typename One<T>::raw x[G::Q], dt[G::Q], z[G::Q], b[G::NB], c[G::NB];
    uint32_t dy[G::Q];
};

// PADDED: some lanes' last states are not there.
template <typename T, int NS, bool PADDED>
__global__ __launch_bounds__(64 * kWaves, 2) void selective_backward_kernel(SelArgs a, SelLayout lay, const float* ends,
                                                                         float* part_bc, float* part_a) {
    typedef SelBack<NS> G;
    constexpr int TT = G::TT, NB = G::NB, Q = G::Q, SUB = G::SUB, SUBS = (int)kSelStateRows / SUB;
    constexpr int P = 16 / NS;  // tokens of a register of sums over channels
    // a lane's own states entering every SUB tokens of a chunk; not its first ones
    // where LDS would hold one workgroup a compute unit in place of two
    constexpr int FIRST = NS <= 8 ? 0 : 1;
    __shared__ float s_h[kWaves][SUBS - FIRST][NS][64];
    // what the rows of a wave hand to each other: step sizes, they times x, and the
    // gradient of what the gate multiplies
    __shared__ f32x4 s_x[kWaves][TT][16];
    __shared__ float s_bc[2][kWaves][2][NB][64];
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Halves halves(k);
    const int per = a.C / a.G, gblk = (int)lay.blocks_bc, nblk = gblk * a.G;
    const int64_t work = lay.places * nblk;
    int buf = 0;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / gblk, block = cb - g * gblk;
        const SelItem e = uniform_item(sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place));
        const int c0 = g * per + (block * kWaves + wave) * kSelChannels + k, end = (g + 1) * per;
        const bool on = c0 < end;
        const int c = on ? c0 : end - 1;  // lanes without a channel: gradients of zero
        const int n = e.seq < 0 ? 0 : (int)e.n;
        const int64_t chan = (int64_t)c * a.N;

        float A[NS], ga[NS], dA[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int s = q * NS + j;
            A[j] = s < a.N ? decay_rate(a.A[chan + s]) : 0.f;
            dA[j] = ga[j] = 0.f;
            if (e.seq < 0 || !on || (PADDED && s >= a.N)) continue;
            if (!e.last) ga[j] = ends[((place + 1) * a.C + c) * (4 * NS) + s];
            else if (a.dfinal && s < a.N) ga[j] = a.dfinal[e.seq * a.C * a.N + chan + s];
        }
        const StepSize step(a.act, c);
        const float D = a.D ? a.D[c] : 0.f;
        float dD = 0.f, dbias = 0.f;

        // at the tile that is loaded next
        typedef RowsOf<TT> Rows;
        const int size = (int)sizeof(T);
        Rows xs(a.x, e.lo, a.x_stride, size, a.C, c, q), dts(a.dt, e.lo, a.dt_stride, size, a.C, c, q);
        Rows zs(a.z, e.lo, a.z_stride, size, a.C, c, q), dys(a.dy, e.lo, a.C, a.y_f32 ? 4 : 2, a.C, c, q);
        StatesOf<T, G> bs(a.B, e.lo, a.b_stride, g * a.N, a.N, q, k), cs(a.Cm, e.lo, a.c_stride, g * a.N, a.N, q, k);
        auto move = [&](int rows) {
            xs.move(rows);
            dts.move(rows);
            dys.move(rows);
            bs.move(rows);
            cs.move(rows);
            if (a.z) zs.move(rows);
        };
        // ALL: or only what the states need
        auto load = [&](int left, auto all, RawBack<T, NS>& r) {
            const TileRows tx = xs.tile(left), td = dts.tile(left);
            bs.load(left, r.b);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                r.x[i] = One<T>::load(tx.r, tx.at(4 * i));
                r.dt[i] = One<T>::load(td.r, td.at(4 * i));
            }
            if (!decltype(all)::value) return;
            const TileRows ty = dys.tile(left), tz = zs.tile(left);
            cs.load(left, r.c);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                r.dy[i] = load_either(ty, 4 * i, a.y_f32);
                if (a.z) r.z[i] = One<T>::load(tz.r, tz.at(4 * i));
            }
        };
        float h[NS];
        // the states over the tile's TT tokens, which are all there
        auto advance = [&](const RawBack<T, NS>& r) {
            float b[NB];
            bs.widen(r.b, b);
            bool wild = false;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float dt = step(One<T>::widen(r.dt[i])), dtx = on ? dt * One<T>::widen(r.x[i]) : 0.f;
                *(f32x2*)&s_x[wave][4 * i + q][k] = f32x2{dt, dtx};
                if (PADDED) wild = wild || !finite(dtx);
            }
            in_wave_order();
            f32x2 next = *(const f32x2*)&s_x[wave][0][k];  // read one token ahead
            unroll<TT>([&](auto token) {
                constexpr int t = decltype(token)::value;
                const f32x2 now = next;
                if (t + 1 < TT) next = *(const f32x2*)&s_x[wave][t + 1 < TT ? t + 1 : 0][k];
                unroll<NS>([&](auto state) {
                    constexpr int j = decltype(state)::value, f = t * NS + j;
                    h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(now[0] * A[j]), h[j],
                                          row_lane<f % 16>(b[f / 16]) * now[1]);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            in_wave_order();
            if (PADDED && __any(wild)) {
                const There<NS> there(a.N, q);
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = there(j, h[j]);
            }
        };
        // What the rows of a wave hand to each other of a tile, `left` tokens of it.  PADDED: whether it is finite.
        float dt[Q];
        auto hand_over = [&](int left, const RawBack<T, NS>& r, auto tail) {
            bool wild = false;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const bool there = on && (!decltype(tail)::value || 4 * i + q < left);
                dt[i] = there ? step(One<T>::widen(r.dt[i])) : 0.f;
                float u = widen_either(r.dy[i], a.y_f32);
                if (a.z) {
                    const float z = One<T>::widen(r.z[i]);
                    u *= z * sigmoid_f(z);
                }
                const f32x4 to = f32x4{dt[i], there ? dt[i] * One<T>::widen(r.x[i]) : 0.f, there ? u : 0.f, 0.f};
                s_x[wave][4 * i + q][k] = to;
                if (PADDED) wild = wild || !finite(to[1]) || !finite(to[2]);
            }
            in_wave_order();
            return !(PADDED && __any(wild));
        };
        // gradients of the tile whose first row of the item is t0, `left` tokens of it, h
        // the states entering it.  TAIL: less than TT of them, or factors that are not finite
        auto tile = [&](int t0, int left, const RawBack<T, NS>& r, auto tail) {
            constexpr bool TAIL = decltype(tail)::value;
            const std::conditional_t<TAIL && PADDED, There<NS>, Everywhere> state_there(a.N, q);
            float b[NB], cc[NB];
            bs.widen(r.b, b);
            cs.widen(r.c, cc);
            if constexpr (!PADDED) hand_over(left, r, tail);
            float before[TT][NS], decay[TT][NS];
            f32x4 next = s_x[wave][0][k];
            __builtin_amdgcn_sched_barrier(0);
            unroll<TT>([&](auto token) {
                constexpr int t = decltype(token)::value;
                const f32x4 here = next;
                if (t + 1 < TT) next = s_x[wave][t + 1 < TT ? t + 1 : 0][k];
                unroll<NS>([&](auto state) {
                    constexpr int j = decltype(state)::value, f = t * NS + j;
                    before[t][j] = h[j];
                    decay[t][j] = 1.f;
                    if (TAIL && t >= left) return;
                    decay[t][j] = state_there(j, __builtin_amdgcn_exp2f(here[0] * A[j]));
                    h[j] = state_there(j, __builtin_fmaf(decay[t][j], h[j], row_lane<f % 16>(b[f / 16]) * here[1]));
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            auto to = [&](void* p, int64_t stride) {
                Rows r(p, e.lo + t0, stride, size, a.C, c, q);
                if (!on) r.lane = kSelNowhere;
                return r.tile(left);
            };
            const TileRows gx = to(a.dx, a.dx_stride), gd = to(a.ddt, a.ddt_stride), gz = to(a.dz, a.dz_stride);
            float pb[NB][P], pc[NB][P];
            next = s_x[wave][TT - 1][k];
            unroll<Q>([&](auto group) {
                constexpr int i = Q - 1 - decltype(group)::value;
                float s[4], ew[4], y[4];
                unroll<4>([&](auto token) {
                    constexpr int t = 3 - decltype(token)::value, at = 4 * i + t, F = at * NS % 16;
                    const f32x4 here = next;
                    if (at > 0) next = s_x[wave][at > 0 ? at - 1 : 0][k];
                    s[t] = ew[t] = y[t] = 0.f;
                    pb[at / P][at % P] = pc[at / P][at % P] = 0.f;
                    if (TAIL && at >= left) return;
                    // h: the states behind this token, ga: the adjoint in front of the next one
                    float vb[NS], vc[NS];
                    add_row<F>(ga, cc[at * NS / 16], here[2]);
#pragma unroll
                    for (int j = 0; j < NS; ++j) ga[j] = state_there(j, ga[j]);
                    y[t] = dot_row<F>(cc[at * NS / 16], h);
                    s[t] = dot_row<F>(b[at * NS / 16], ga);
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        vc[j] = here[2] * h[j];
                        vb[j] = ga[j] * here[1];
                        ga[j] *= decay[at][j];
                        const float wn = ga[j] * before[at][j];
                        ew[t] = __builtin_fmaf(wn, A[j], ew[t]);
                        dA[j] = __builtin_fmaf(wn, here[0], dA[j]);
                        h[j] = before[at][j];
                    }
                    join_states<NS>(vb, vc, halves, pb[at / P][at % P], pc[at / P][at % P]);
                    __builtin_amdgcn_sched_barrier(0);
                });
                const bool there = on && (!TAIL || 4 * i + q < left);
                const float S = sum_rows(s), E = sum_rows(ew) * kLn2;
                const float x = there ? One<T>::widen(r.x[i]) : 0.f, dy = there ? widen_either(r.dy[i], a.y_f32) : 0.f;
                float u = dy, dz = 0.f;
                if (a.z) {
                    const float z = there ? One<T>::widen(r.z[i]) : 0.f, sg = sigmoid_f(z);
                    u *= z * sg;
                    float p = sum_rows(y);
                    if (a.D) p = __builtin_fmaf(D, x, p);
                    dz = dy * p * (sg * (1.f + z * (1.f - sg)));
                }
                float dx = dt[i] * S;
                if (a.D) dx = __builtin_fmaf(D, u, dx);  // not 0 times an infinite u
                const float slope = step.slope(One<T>::widen(r.dt[i]), dt[i]);
                float draw = there ? (x * S + E) * slope : 0.f;
                if (step.cut && slope == 0.f) draw = 0.f;  // of an infinite gradient, too
                dbias += draw;
                dD += u * x;
                One<T>::store(gx.r, gx.at(4 * i), dx);
                One<T>::store(gd.r, gd.at(4 * i), draw);
                if (a.z) One<T>::store(gz.r, gz.at(4 * i), dz);
                // the sums over the wave's channels of the registers that are complete
                unroll<NB>([&](auto reg) {
                    constexpr int o = decltype(reg)::value;
                    if constexpr (P * o >= 4 * i && P * o < 4 * i + 4) {
                        s_bc[buf][wave][0][o][lane] = join_tokens<NS>(pb[o], halves);
                        s_bc[buf][wave][1][o][lane] = join_tokens<NS>(pc[o], halves);
                    }
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            // and over the workgroup's.  Only LDS is waited for: a barrier of the usual kind
            // would also wait until the gradients just stored are in memory.
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            for (int o = threadIdx.x; o < 2 * NB * 64; o += 64 * kWaves) {
                const int l = o & 63, i = (o >> 6) % NB, which = (o >> 6) / NB;
                const int s = (l >> 4) * NS + joined_state<NS>(l & 15), t = P * i + joined_token<NS>(l & 15);
                if (t >= left || s >= a.N) continue;
                float v = 0.f;
#pragma unroll
                for (int o2 = 0; o2 < kWaves; ++o2) v += s_bc[buf][o2][which][i][l];
                part_bc[(((int64_t)block * a.T + e.lo + t0 + t) * a.G + g) * (2 * a.N) + which * a.N + s] = v;
            }
            buf ^= 1;  // the readers of this one are done before the barrier after the next
        };
        int chunk = n > 0 ? (n - 1) / (int)kSelStateRows * (int)kSelStateRows : -1;
        if (chunk > 0) move(chunk);
        for (; chunk >= 0; chunk -= (int)kSelStateRows) {
            const int64_t slot = sel_place(a.cu != nullptr, e.seq, e.first, a.L, kSelStateRows) +
                                 (e.index * lay.item + chunk) / kSelStateRows;
            const float* saved = a.states_in + slot * a.C * a.N + chan;
            const int here = min(n - chunk, (int)kSelStateRows), subs = (here + SUB - 1) / SUB, ahead = (subs - 1) * SUB;
            RawBack<T, NS> cur, nxt;
            auto enter = [&] {
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const int s = q * NS + j;
                    h[j] = on && s < a.N ? saved[s] : 0.f;
                }
            };
            auto keep = [&](int t) {  // the states entering token t of the chunk
                if (t % SUB || t / SUB < FIRST) return;
#pragma unroll
                for (int j = 0; j < NS; ++j) s_h[wave][t / SUB - FIRST][j][lane] = h[j];
            };
            enter();
            constexpr int AHEAD = (SUBS - 1) * SUB / TT;  // tiles in front of a whole chunk's last SUB tokens
            if (AHEAD <= 7 && subs == SUBS) {
                // all of them in flight at once: the registers of a tile's states are still free
                RawBack<T, NS> raw[AHEAD];
                unroll<AHEAD>([&](auto o) {
                    load(TT, std::false_type{}, raw[decltype(o)::value]);
                    move(TT);
                });
                unroll<AHEAD>([&](auto o) {
                    keep(decltype(o)::value * TT);
                    advance(raw[decltype(o)::value]);
                });
            } else {
                if (ahead) {
                    load(TT, std::false_type{}, nxt);
                    move(TT);
                }
                for (int t = 0; t < ahead; t += TT) {
                    cur = nxt;
                    if (t + TT < ahead) {
                        load(TT, std::false_type{}, nxt);
                        move(TT);
                    }
                    keep(t);
                    advance(cur);
                }
            }
            keep(ahead);
            int t = (here - 1) / TT * TT;
            if (SUB > TT) move(t - ahead);
            load(here - t, std::true_type{}, nxt);
            for (; t >= 0; t -= TT) {
                cur = nxt;
                move(-TT);
                if (t) load(TT, std::true_type{}, nxt);
                if (t / SUB < FIRST) {
                    enter();
                } else {
#pragma unroll
                    for (int j = 0; j < NS; ++j) h[j] = s_h[wave][t / SUB - FIRST][j][lane];
                }
                if constexpr (SUB > TT) {  // from the state in LDS to this tile
                    const int skip = t % SUB;
                    move(TT - skip);
                    for (int o = 0; o < skip; o += TT) {
                        RawBack<T, NS> part;
                        load(TT, std::false_type{}, part);
                        move(TT);
                        advance(part);
                    }
                    move(-TT);
                }
                const bool whole = t + TT <= here;
                if constexpr (PADDED) {
                    const bool tame = whole ? hand_over(TT, cur, std::false_type{}) : hand_over(here - t, cur, std::true_type{});
                    if (whole && tame) tile(chunk + t, TT, cur, std::false_type{});
                    else tile(chunk + t, min(here - t, TT), cur, std::true_type{});
                } else {
                    if (whole) tile(chunk + t, TT, cur, std::false_type{});
                    else tile(chunk + t, here - t, cur, std::true_type{});
                }
            }
            move(TT - (int)kSelStateRows);
        }
        dD = sum_all_rows(dD);
        dbias = sum_all_rows(dbias);
        float* part = part_a + place * a.C * (a.N + 2);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int s = q * NS + j;
            if (!on || s >= a.N) continue;
            part[chan + s] = dA[j];
            if (e.seq >= 0 && e.index == 0 && a.dinit) a.dinit[e.seq * a.C * a.N + chan + s] = ga[j];
        }
        if (on && q == 0) {
            part[(int64_t)a.C * a.N + c] = dD;
            part[(int64_t)a.C * (a.N + 1) + c] = dbias;
        }
    }
}

// ---------------------------------------------------------------- sums
// dB and dC from the channel blocks' sums.
template <typename T>
__global__ __launch_bounds__(256) void selective_sum_bc_kernel(SelArgs a, const float* part, int64_t blocks) {
    const RowRange live = live_rows(a.cu, a.nseq, a.T);
    const int width = a.G * 2 * a.N;
    const int64_t end = live.hi * width;
    for (int64_t i = live.lo * width + (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (int64_t)gridDim.x * 256) {
        float v = 0.f;
#pragma unroll 8
        for (int64_t b = 0; b < blocks; ++b) v += part[b * a.T * width + i];
        const int64_t row = i / width;
        const int at = (int)(i - row * width), g = at / (2 * a.N), s = at - g * 2 * a.N;
        if (s < a.N) ((T*)a.dB)[row * a.db_stride + g * a.N + s] = (T)v;
        else ((T*)a.dC)[row * a.dc_stride + g * a.N + s - a.N] = (T)v;
    }
}

// dA, dD and dbias from the items' sums.
__global__ __launch_bounds__(kSumThreads) void selective_sum_kernel(SelArgs a, const float* part, int64_t places) {
    const int64_t width = (int64_t)a.C * (a.N + 2), states = (int64_t)a.C * a.N;
    for (int64_t b = blockIdx.x; b < (width + kSumCols - 1) / kSumCols; b += gridDim.x) {
        const int64_t col = b * kSumCols + threadIdx.x % kSumCols;
        const float v = column_sum(places, [&](int64_t t) { return col < width ? part[t * width + col] : 0.f; });
        __syncthreads();  // the sums of the columns before have been read
        if (threadIdx.x >= kSumCols || col >= width) continue;
        if (col < states) a.dA[col] = v;
        else if (col < states + a.C) {
            if (a.dD) a.dD[col - states] = v;
        } else if (a.dbias) a.dbias[col - states - a.C] = v;
    }
}

template <typename T, int NS>
hipError_t run_backward(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    float* ends = (float*)((char*)ws + lay.states);
    float* steps = (float*)((char*)ws + lay.steps);
    float* part_bc = (float*)((char*)ws + lay.part_bc);
    float* part_a = (float*)((char*)ws + lay.part_a);
    const int per = a.C / a.G;
    hipError_t e = hipSuccess;
    if (lay.places > 0) {
        if (!lay.whole) {
            const int64_t work = lay.places * ((per + 4 * kSelChannels - 1) / (4 * kSelChannels)) * a.G;
            hipLaunchKernelGGL((selective_adjoint_kernel<T, NS>), dim3((unsigned)std::min<int64_t>(work, kMaxBlocks)),
                               dim3(256), 0, stream, a, lay, ends, steps);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            const int64_t blocks = ((int64_t)a.C * 4 * NS + 255) / 256 * a.nseq;
            hipLaunchKernelGGL(selective_carry_back_kernel, dim3((unsigned)std::min<int64_t>(blocks, kMaxBlocks)),
                               dim3(256), 0, stream, a, lay, ends, steps, 4 * NS);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        const int64_t work = lay.places * lay.blocks_bc * a.G;
        const dim3 grid((unsigned)std::min<int64_t>(work, kMaxBlocks)), block(64 * kWaves);
        if (a.N == 4 * NS)
            hipLaunchKernelGGL((selective_backward_kernel<T, NS, false>), grid, block, 0, stream, a, lay, ends, part_bc, part_a);
        else
            hipLaunchKernelGGL((selective_backward_kernel<T, NS, true>), grid, block, 0, stream, a, lay, ends, part_bc, part_a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.T > 0) {
            const int64_t elements = a.T * a.G * 2 * a.N;
            hipLaunchKernelGGL((selective_sum_bc_kernel<T>),
                               dim3((unsigned)std::min<int64_t>((elements + 255) / 256, 1 << 16)), dim3(256), 0, stream,
                               a, part_bc, lay.blocks_bc);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    const int64_t blocks = ((int64_t)a.C * (a.N + 2) + kSumCols - 1) / kSumCols;
    hipLaunchKernelGGL(selective_sum_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 16)), dim3(kSumThreads), 0,
                       stream, a, part_a, lay.places);
    return hipGetLastError();
}

template <typename T>
hipError_t by_states(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    if (a.N <= 4) return run_backward<T, 1>(a, lay, ws, stream);
    if (a.N <= 8) return run_backward<T, 2>(a, lay, ws, stream);
    if (a.N <= 16) return run_backward<T, 4>(a, lay, ws, stream);
    if (a.N <= 32) return run_backward<T, 8>(a, lay, ws, stream);
    return run_backward<T, 16>(a, lay, ws, stream);
}

}  // namespace

hipError_t launch_selective_backward(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    return a.dtype == 1 ? by_states<bf16_t>(a, lay, ws, stream) : by_states<float>(a, lay, ws, stream);
}

}  // namespace ssd
