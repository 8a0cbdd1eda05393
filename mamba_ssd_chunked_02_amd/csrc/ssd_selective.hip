// Selective scan on gfx950: per channel c, state n and token t
//   h = exp(dt A[c, n]) h + dt x B[t, n],   y = (sum_n h C[t, n] + D[c] x) silu(z)
// with the step size dt of a (token, channel) from its raw value.
//
// A long sequence is cut into items, so that there are waves enough: a first launch
// takes every item but a sequence's last from a state of zero to the state it ends
// with and the sum S of its step sizes, a second carries the states over the items
// (an item multiplies the state entering it by exp(A S)), a third writes y.  Where
// the sequences alone fill the chip only the third runs.
//
// At 16 states the vector ALU bounds it, not HBM: 8.3 instructions a (token, channel,
// state) here and 5.5 in the first launch, of which the exponential takes 8.4 cycles a
// wave, its argument's product, the state's and y's 4 to 4.6 each.  Some are the
// compiler's: of 281 vector instructions in the loop over tiles 24 are moves and 9 lane
// reads of spilled scalars; the bf16 kernels for up to 4 states also keep 3 to 5
// registers in scratch.  Packed 49152 x 8192 x 16, bf16: y 1.58 to 1.67 ms (2.6 GB read,
// 0.86 written), the end states 1.06 to 1.12; 8 x 2048 x 5120 x 16 as a whole 540 us,
// 2.5 T states a second where 8 waves a SIMD reach 3.7: 2560 waves on 1024 SIMDs.  A
// wave's lanes are 16 channels by four quarters of the states: by channel alone a lane
// would need 16 states, 64 channels' waves and so four times the items, by state alone
// every load would serve one channel.
#include <algorithm>
#include <type_traits>

#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kWaves = 4;                            // of a workgroup
constexpr int kBlockChannels = kWaves * kSelChannels;
constexpr int64_t kMaxBlocks = 1 << 22;              // a launch counts its lanes in 32 bits

template <typename T, int NS>
struct RawTile {
    typedef SelTile<NS> G;
    typename One<T>::raw x[G::Q], dt[G::Q], z[G::Q], b[G::NB], c[G::NB];
};

// LOCAL: the states that items end with, from zero.  Else y, final and saved states.
// PADDED: some lanes' last states are not there (11 states, 8 x 2048 x 5120: 535 us, 505
// without looking after them; chosen by a branch in front of each tile 570 to 595).
template <typename T, int NS, bool LOCAL, bool PADDED>
__global__ __launch_bounds__(64 * kWaves, NS <= 4 ? 6 : 4) void selective_kernel(SelArgs a, SelLayout lay, float* ends, float* steps) {
    typedef SelTile<NS> G;
    constexpr int TT = G::TT, NB = G::NB, Q = G::Q;
    // what the rows of a wave hand to each other: step sizes, and they times x
    __shared__ float s_x[kWaves][TT][16][2];
    __shared__ float s_h[PADDED ? kWaves : 1][NS][64];  // the states entering a tile
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = a.C / a.G, nblk = (per + kBlockChannels - 1) / kBlockChannels * a.G;
    const int64_t work = lay.places * nblk;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / (nblk / a.G);
        const SelItem e = uniform_item(sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place));
        if (e.seq < 0 || (LOCAL && e.last)) continue;
        const int c0 = g * per + (cb - g * (nblk / a.G)) * kBlockChannels + wave * kSelChannels, end = (g + 1) * per;
        if (c0 >= end) continue;
        const bool on = c0 + k < end;
        const int c = on ? c0 + k : end - 1;  // lanes without a channel take the last one's, and write nothing
        const int n = (int)e.n;
        const int64_t chan = (int64_t)c * a.N;

        float A[NS], h[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int s = q * NS + j;
            const bool there = s < a.N;
            A[j] = there ? decay_rate(a.A[chan + s]) : 0.f;
            h[j] = 0.f;
            if (LOCAL) continue;
            if (PADDED && !there) continue;
            if (e.index > 0) h[j] = ends[((place - 1) * a.C + c) * (4 * NS) + s];
            else if (a.init && there) h[j] = a.init[e.seq * a.C * a.N + chan + s];
        }
        const StepSize step(a.act, c);
        const float D = !LOCAL && a.D ? a.D[c] : 0.f;
        float total = 0.f;
        uint32_t decays = q == 0 ? 0 : ~0u;  // LOCAL: the first token has nothing to decay, be its factor infinite

        const bool gated = !LOCAL && a.z;
        typedef RowsOf<TT> Rows;
        const int size = (int)sizeof(T), ysize = a.y_f32 ? 4 : 2;
        Rows xs(a.x, e.lo, a.x_stride, size, a.C, c, q), dts(a.dt, e.lo, a.dt_stride, size, a.C, c, q);
        Rows zs(a.z, e.lo, a.z_stride, size, a.C, c, q), ys(a.y, e.lo, a.C, ysize, a.C, c, q);
        if (!on) ys.lane = kSelNowhere;
        StatesOf<T, G> bs(a.B, e.lo, a.b_stride, g * a.N, a.N, q, k), cs(a.Cm, e.lo, a.c_stride, g * a.N, a.N, q, k);
        // the next tile, of which `left` tokens are there
        auto load = [&](int left, RawTile<T, NS>& r) {
            const TileRows tx = xs.tile(left), td = dts.tile(left);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                r.x[i] = One<T>::load(tx.r, tx.at(4 * i));
                r.dt[i] = One<T>::load(td.r, td.at(4 * i));
            }
            bs.load(left, r.b);
            xs.move(TT);
            dts.move(TT);
            bs.move(TT);
            if constexpr (LOCAL) return;
            cs.load(left, r.c);
            cs.move(TT);
            if (!gated) return;
            const TileRows tz = zs.tile(left);
#pragma unroll
            for (int i = 0; i < Q; ++i) r.z[i] = One<T>::load(tz.r, tz.at(4 * i));
            zs.move(TT);
        };
        // the tile's first `left` tokens; a row behind them takes a step of 0
        auto tile = [&](int left, const RawTile<T, NS>& r) {
            float b[NB], cc[NB];
            bs.widen(r.b, b);
            if (!LOCAL) cs.widen(r.c, cc);
            const TileRows ty = ys.tile(left);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                float dt = step(One<T>::widen(r.dt[i]));
                if (left < TT) dt = 4 * i + q < left ? dt : 0.f;
                if (LOCAL) total += dt;
                const float dtx = dt * One<T>::widen(r.x[i]);
                if (LOCAL && i == 0) dt = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, dt) & decays);
                *(f32x2*)s_x[wave][4 * i + q][k] = f32x2{dt, dtx};
            }
            if constexpr (PADDED) {
#pragma unroll
                for (int j = 0; j < NS; ++j) s_h[wave][j][lane] = h[j];
            }
            in_wave_order();
            auto tokens = [&](auto careful) {
                const std::conditional_t<decltype(careful)::value, There<NS>, Everywhere> there(a.N, q);
                f32x2 next = *(const f32x2*)s_x[wave][0][k];
                unroll<Q>([&](auto group) {
                    constexpr int i = decltype(group)::value;
                    float y[4];
                    unroll<4>([&](auto token) {
                        constexpr int t = decltype(token)::value, at = 4 * i + t;
                        const f32x2 now = next;  // read one token ahead
                        if (at + 1 < TT) next = *(const f32x2*)s_x[wave][at + 1 < TT ? at + 1 : 0][k];
                        unroll<NS>([&](auto state) {
                            constexpr int j = decltype(state)::value, f = at * NS + j;
                            h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(now[0] * A[j]), h[j],
                                                  row_lane<f % 16>(b[f / 16]) * now[1]);
                            h[j] = there(j, h[j]);
                        });
                        if constexpr (!LOCAL) y[t] = dot_row<at * NS % 16>(cc[at * NS / 16], h);
                    });
                    if constexpr (!LOCAL) {
                        float v = sum_rows(y);
                        if (a.D) v = __builtin_fmaf(D, One<T>::widen(r.x[i]), v);  // not 0 times an infinite x
                        if (gated) {
                            const float z = One<T>::widen(r.z[i]);
                            v *= z * sigmoid_f(z);
                        }
                        if (a.y_f32) One<float>::store(ty.r, ty.at(4 * i), v);
                        else One<bf16_t>::store(ty.r, ty.at(4 * i), v);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                });
            };
            tokens(std::false_type{});
            if constexpr (PADDED) {
                // the last of them, which is as the others are: 0, or NaN from some token on
                if (__any(q == 3 && !(h[NS - 1] == 0.f))) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) h[j] = s_h[wave][j][lane];
                    tokens(std::true_type{});
                }
            }
            in_wave_order();
            decays = ~0u;
            if (!LOCAL) ys.move(TT);
        };
        RawTile<T, NS> cur, nxt;
        if (n > 0) load(n, nxt);
        for (int t0 = 0; t0 < n; t0 += TT) {
            cur = nxt;
            if (t0 + TT < n) load(n - t0 - TT, nxt);
            if (!LOCAL && a.states_out && t0 % kSelStateRows == 0 && on) {
                const int64_t at = sel_place(a.cu != nullptr, e.seq, e.first, a.L, kSelStateRows) +
                                   (e.index * lay.item + t0) / kSelStateRows;
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    if (q * NS + j < a.N) a.states_out[at * a.C * a.N + chan + q * NS + j] = h[j];
            }
            tile(n - t0, cur);
        }
        if constexpr (LOCAL) {
            total = sum_all_rows(total);
            if (on) {
#pragma unroll
                for (int j = 0; j < NS; ++j) ends[(place * a.C + c) * (4 * NS) + q * NS + j] = h[j];
                if (q == 0) steps[place * a.C + c] = total;
            }
        } else if (e.last && a.final_state && on) {
#pragma unroll
            for (int j = 0; j < NS; ++j)
                if (q * NS + j < a.N) a.final_state[e.seq * a.C * a.N + chan + q * NS + j] = h[j];
        }
    }
}

// Carries the states over the items of a sequence, in place: what an item ends
// with from zero becomes what it ends with.
__global__ __launch_bounds__(256) void selective_carry_kernel(SelArgs a, SelLayout lay, float* ends, const float* steps,
                                                              int padded) {
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
        const float h = a.init && there ? a.init[(s * a.C + c) * a.N + n] : 0.f;
        const int64_t place = sel_place(a.cu != nullptr, s, r.lo, a.L, lay.item);
        carry(ends + place * row + at, row, steps + place * a.C + c, a.C, items - 1, A, h);
    }
}

// ------------------------------------------------------------------ one token
// A few operations per byte of state: HBM, from a few MB of states on.  Four lanes a
// channel, lane q of them the states 4 q .. 4 q + 3 of every sixteen; a lane takes
// kStepRows sequences, so that their states are in flight together and A is read once
// for them.  256 x 5120 x 16: 35 us, 176 MB, 5.0 TB/s; one
// sequence of 1536 channels 4.7 us, which is a launch and one access' latency.
// VEC: states by fours, and A, B and C aligned to them.
constexpr int kStepRows = 4;

template <typename T>
struct Four;
template <>
struct Four<float> {
    __device__ static inline f32x4 load(const float* p) { return *(const f32x4*)p; }
};
template <>
struct Four<bf16_t> {
    __device__ static inline f32x4 load(const bf16_t* p) { return Raw<bf16_t>::widen(*(const Raw<bf16_t>::type*)p); }
};
template <typename T, bool VEC>
__device__ inline f32x4 four_of(const T* p, int n, int N) {
    if constexpr (VEC) return Four<T>::load(p + n);
    f32x4 v = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < N) v[j] = One<T>::widen(One<T>::load(p + n + j));
    return v;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void selective_step_kernel(SelArgs a, const float* state, float* state_out) {
    const int q = threadIdx.x & 3, blocks = (a.C + 63) / 64;
    const int64_t groups = (a.nseq + kStepRows - 1) / kStepRows;
    for (int64_t w = blockIdx.x; w < groups * blocks; w += gridDim.x) {
        const int64_t s0 = w / blocks * kStepRows;
        const int c = (int)(w % blocks) * 64 + (threadIdx.x >> 2);
        if (c >= a.C) continue;  // the four lanes of a channel together
        const int rows = (int)min(a.nseq - s0, (int64_t)kStepRows);
        const int64_t first = (int64_t)(c / (a.C / a.G)) * a.N;  // of the channel's group
        const StepSize step(a.act, c);
        float x[kStepRows], dt[kStepRows], z[kStepRows], y[kStepRows];
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            const int64_t s = s0 + min(r, rows - 1);
            x[r] = One<T>::widen(One<T>::load((const T*)a.x + s * a.x_stride + c));
            dt[r] = One<T>::widen(One<T>::load((const T*)a.dt + s * a.dt_stride + c));
            z[r] = a.z ? One<T>::widen(One<T>::load((const T*)a.z + s * a.z_stride + c)) : 0.f;
            y[r] = 0.f;
        }
        const float D = a.D ? a.D[c] : 0.f;
        for (int n = 4 * q; n < a.N; n += 16) {
            f32x4 A = four_of<float, VEC>(a.A + (int64_t)c * a.N, n, a.N), h[kStepRows], B[kStepRows], C[kStepRows];
#pragma unroll
            for (int r = 0; r < kStepRows; ++r) {
                const int64_t s = s0 + min(r, rows - 1), at = (s * a.C + c) * a.N;
                h[r] = four_of<float, VEC>(state + at, n, a.N);
                B[r] = four_of<T, VEC>((const T*)a.B + s * a.b_stride + first, n, a.N);
                C[r] = four_of<T, VEC>((const T*)a.Cm + s * a.c_stride + first, n, a.N);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) A[j] = decay_rate(A[j]);
#pragma unroll
            for (int r = 0; r < kStepRows; ++r) {
                if (r >= rows) break;
                const float d = step(dt[r]), xs = d * x[r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[r][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A[j]), h[r][j], B[r][j] * xs);
                    if (VEC || n + j < a.N) y[r] = __builtin_fmaf(C[r][j], h[r][j], y[r]);
                }
                float* to = state_out + ((s0 + r) * a.C + c) * a.N + n;
                if constexpr (VEC) {
                    *(f32x4*)to = h[r];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < a.N) to[j] = h[r][j];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kStepRows; ++r) {
            float v = y[r];
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            if (a.D) v += D * x[r];
            if (a.z) v *= z[r] * sigmoid_f(z[r]);
            if (q != 0 || r >= rows) continue;
            if (a.y_f32) ((float*)a.y)[(s0 + r) * a.C + c] = v;
            else ((bf16_t*)a.y)[(s0 + r) * a.C + c] = (bf16_t)v;
        }
    }
}

template <typename T, int NS>
hipError_t run_scan(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    float* ends = (float*)((char*)ws + lay.states);
    float* steps = (float*)((char*)ws + lay.steps);
    const int per = a.C / a.G;
    const int64_t work = lay.places * ((per + kBlockChannels - 1) / kBlockChannels) * a.G;
    if (work == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>(work, kMaxBlocks)), block(64 * kWaves);
    if (!lay.whole) {
        hipLaunchKernelGGL((selective_kernel<T, NS, true, false>), grid, block, 0, stream, a, lay, ends, steps);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t blocks = ((int64_t)a.C * 4 * NS + 255) / 256 * a.nseq;
        hipLaunchKernelGGL(selective_carry_kernel, dim3((unsigned)std::min<int64_t>(blocks, kMaxBlocks)), dim3(256), 0,
                           stream, a, lay, ends, steps, 4 * NS);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.N == 4 * NS)
        hipLaunchKernelGGL((selective_kernel<T, NS, false, false>), grid, block, 0, stream, a, lay, ends, steps);
    else
        hipLaunchKernelGGL((selective_kernel<T, NS, false, true>), grid, block, 0, stream, a, lay, ends, steps);
    return hipGetLastError();
}

template <typename T>
hipError_t by_states(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    if (a.N <= 4) return run_scan<T, 1>(a, lay, ws, stream);
    if (a.N <= 8) return run_scan<T, 2>(a, lay, ws, stream);
    if (a.N <= 16) return run_scan<T, 4>(a, lay, ws, stream);
    if (a.N <= 32) return run_scan<T, 8>(a, lay, ws, stream);
    return run_scan<T, 16>(a, lay, ws, stream);
}

}  // namespace

hipError_t launch_selective_scan(const SelArgs& a, const SelLayout& lay, void* ws, hipStream_t stream) {
    return a.dtype == 1 ? by_states<bf16_t>(a, lay, ws, stream) : by_states<float>(a, lay, ws, stream);
}

hipError_t launch_selective_step(const SelArgs& a, const float* state, float* state_out, hipStream_t stream) {
    const int64_t work = (a.nseq + kStepRows - 1) / kStepRows * ((a.C + 63) / 64);
    if (work == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>(work, kMaxBlocks)), block(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, state, state_out); };
    const uintptr_t four = a.dtype == 1 ? 8 : 16;
    const bool vec = a.N % 4 == 0 && (uintptr_t)a.A % 16 == 0 && (uintptr_t)a.B % four == 0 && (uintptr_t)a.Cm % four == 0 &&
                     a.b_stride % 4 == 0 && a.c_stride % 4 == 0;
    if (a.dtype == 1) vec ? go(selective_step_kernel<bf16_t, true>) : go(selective_step_kernel<bf16_t, false>);
    else vec ? go(selective_step_kernel<float, true>) : go(selective_step_kernel<float, false>);
    return hipGetLastError();
}

int64_t sel_saved_states(bool packed, int64_t nseq, int64_t L, int64_t T) {
    return sel_places(packed, nseq, L, T, kSelStateRows);
}

SelLayout sel_layout(const SelArgs& a, bool backward) {
    SelLayout l = {};
    const int64_t waves = (a.C + kSelChannels - 1) / kSelChannels;
    const int padded = a.N <= 4 ? 4 : a.N <= 8 ? 8 : a.N <= 16 ? 16 : a.N <= 32 ? 32 : 64;
    auto up = [](int64_t v) { return std::max<int64_t>((v + kSelStateRows - 1) / kSelStateRows, 1) * kSelStateRows; };
    // Forward: sequences of one length that bring 2 waves a SIMD go as a whole (8 x 2048 x
    // 5120 forward and backward 2.48 ms; cut into 512 tokens forward 2.54), else items for 16
    // waves a SIMD, so that their unequal ends even out (packed 49152 x 8192: 512 and 1024
    // tokens 2.65 ms, 1536, which the rule takes, 2.66, 2048 2.68, 6144 3.07), but 128 tokens
    // at least (4096 x 1536: 64 and 128 tokens 69 us, 256 91; 64 take twice the workspace).
    // Backward: always items, since no sequence count that is common fills two waves a SIMD
    // evenly (8 x 2048 x 5120 forward and backward 2.48 ms, whole 2.79).
    const int64_t least = backward ? 64 : 128;
    if (!backward && !a.cu && a.nseq * waves >= 2048) l.item = up(a.L);
    else l.item = std::max(least, up((int64_t)((double)a.T * waves / 16384)));
    l.places = sel_places(a.cu != nullptr, a.nseq, a.L, a.T, l.item);
    l.whole = !a.cu ? l.item >= a.L : l.item >= a.T;
    size_t at = 0;
    auto region = [&at](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (!l.whole) {
        l.states = region((size_t)l.places * a.C * padded * 4);
        l.steps = region((size_t)l.places * a.C * 4);
    }
    if (backward) {
        const int per = a.C / a.G;
        l.blocks_bc = (per + kSelBackChannels - 1) / kSelBackChannels;
        l.part_bc = region((size_t)l.blocks_bc * a.T * a.G * 2 * a.N * 4);
        l.part_a = region((size_t)l.places * a.C * (a.N + 2) * 4);
    }
    l.total = at;
    return l;
}

}  // namespace ssd
