// Selective scan on gfx950: per channel c, state n and token t
//   h = exp(dt A[c, n]) h + dt x B[t, n],   y = (sum_n h C[t, n] + D[c] x) silu(z)
// with the step size dt of a (token, channel) from its raw value.
//
// A long sequence is cut into items, so that there are waves enough: a first launch
// takes every item but a sequence's last from a state of zero to the state it ends
// with and the sum S of its step sizes, a second carries the states over the items
// (an item multiplies the state entering it by exp(A S)), a third writes y.  Where
// the sequences alone fill the chip only the third runs.
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
template <typename T, int NS, bool LOCAL>
__global__ __launch_bounds__(64 * kWaves) void selective_kernel(SelArgs a, SelLayout lay, float* ends, float* steps) {
    typedef SelTile<NS> G;
    constexpr int TT = G::TT, NB = G::NB, Q = G::Q;
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = a.C / a.G, nblk = (per + kBlockChannels - 1) / kBlockChannels * a.G;
    const int64_t work = lay.places * nblk;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / (nblk / a.G);
        const SelItem e = sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place);
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
            A[j] = there ? a.A[chan + s] * kLog2e : 0.f;
            h[j] = 0.f;
            if (LOCAL) continue;
            if (e.index > 0) h[j] = ends[((place - 1) * a.C + c) * (4 * NS) + s];
            else if (a.init && there) h[j] = a.init[e.seq * a.C * a.N + chan + s];
        }
        const StepSize step(a.act, c);
        const float D = !LOCAL && a.D ? a.D[c] : 0.f;
        float total = 0.f;

        const T* xp = (const T*)a.x + e.lo * a.x_stride + c;
        const T* dp = (const T*)a.dt + e.lo * a.dt_stride + c;
        const T* zp = (const T*)a.z + e.lo * a.z_stride + c;
        const T* bp = (const T*)a.B + e.lo * a.b_stride + g * a.N;
        const T* cp = (const T*)a.Cm + e.lo * a.c_stride + g * a.N;
        const bool gated = !LOCAL && a.z;
        auto load = [&](int t0, RawTile<T, NS>& r) {
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int64_t t = min(t0 + 4 * i + q, n - 1);
                r.x[i] = One<T>::load(xp + t * a.x_stride);
                r.dt[i] = One<T>::load(dp + t * a.dt_stride);
                if (gated) r.z[i] = One<T>::load(zp + t * a.z_stride);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int f = 16 * i + k, s = min(q * NS + f % NS, a.N - 1);
                const int64_t t = min(t0 + f / NS, n - 1);
                r.b[i] = One<T>::load(bp + t * a.b_stride + s);
                if (!LOCAL) r.c[i] = One<T>::load(cp + t * a.c_stride + s);
            }
        };
        // TAIL: only some of the tile's tokens are there
        auto tile = [&](int t0, const RawTile<T, NS>& r, auto tail) {
            constexpr bool TAIL = decltype(tail)::value;
            float b[NB], cc[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int f = 16 * i + k;
                const bool there = q * NS + f % NS < a.N && (!TAIL || t0 + f / NS < n);
                b[i] = there ? One<T>::widen(r.b[i]) : 0.f;
                cc[i] = !LOCAL && there ? One<T>::widen(r.c[i]) : 0.f;
            }
            unroll<Q>([&](auto group) {
                constexpr int i = decltype(group)::value;
                if (TAIL && t0 + 4 * i >= n) return;
                const bool there = !TAIL || t0 + 4 * i + q < n;
                const float x = One<T>::widen(r.x[i]), dt = there ? step(One<T>::widen(r.dt[i])) : 0.f;
                if (LOCAL) total += dt;
                float dts[4], xs[4], y[4];
                rows_to_all(dt, dts);
                rows_to_all(there ? dt * x : 0.f, xs);
                unroll<4>([&](auto token) {
                    constexpr int t = decltype(token)::value;
                    const bool live = !TAIL || t0 + 4 * i + t < n;
                    y[t] = 0.f;
                    unroll<NS>([&](auto state) {
                        constexpr int j = decltype(state)::value, f = (4 * i + t) * NS + j;
                        const float d = __builtin_amdgcn_exp2f(dts[t] * A[j]);
                        h[j] = __builtin_fmaf(live ? d : 1.f, h[j], row_lane<f % 16>(b[f / 16]) * xs[t]);
                        if (!LOCAL) y[t] = __builtin_fmaf(row_lane<f % 16>(cc[f / 16]), h[j], y[t]);
                    });
                });
                if constexpr (!LOCAL) {
                    float v = sum_rows(y) + D * x;
                    if (gated) {
                        const float z = One<T>::widen(r.z[i]);
                        v *= z * sigmoid_f(z);
                    }
                    if (on && there) store_one(a.y, (e.lo + t0 + 4 * i + q) * a.C + c, a.y_f32, v);
                }
            });
        };
        RawTile<T, NS> cur, nxt;
        if (n > 0) load(0, nxt);
        for (int t0 = 0; t0 < n; t0 += TT) {
            cur = nxt;
            if (t0 + TT < n) load(t0 + TT, nxt);
            if (!LOCAL && a.states_out && t0 % kSelStateRows == 0 && on) {
                const int64_t at = sel_place(a.cu != nullptr, e.seq, e.first, a.L, kSelStateRows) +
                                   (e.index * lay.item + t0) / kSelStateRows;
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    if (q * NS + j < a.N) a.states_out[at * a.C * a.N + chan + q * NS + j] = h[j];
            }
            if (t0 + TT <= n) tile(t0, cur, std::false_type{});
            else tile(t0, cur, std::true_type{});
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
        const float A = there ? a.A[(int64_t)c * a.N + n] * kLog2e : 0.f;
        float h = a.init && there ? a.init[(s * a.C + c) * a.N + n] : 0.f;
        const int64_t place = sel_place(a.cu != nullptr, s, r.lo, a.L, lay.item);
        float* p = ends + place * row + at;
        const float* st = steps + place * a.C + c;
        for (int64_t j = 0; j < items - 1; ++j, p += row, st += a.C) {
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * *st), h, *p);
            *p = h;
        }
    }
}

// ------------------------------------------------------------------ one token
// Four lanes a channel, lane q of them the states q, q + 4, ... (VEC: 4 q + 0..3,
// then 16 more, read as one vector); a few operations per byte of state: HBM.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void selective_step_kernel(SelArgs a, const float* state, float* state_out) {
    const int64_t total = a.nseq * a.C;
    const int q = threadIdx.x & 3, per = a.C / a.G;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 2; i < total; i += (int64_t)gridDim.x * 64) {
        const int64_t s = i / a.C;
        const int c = (int)(i - s * a.C);
        const float x = One<T>::widen(One<T>::load((const T*)a.x + s * a.x_stride + c));
        const float dt = StepSize(a.act, c)(One<T>::widen(One<T>::load((const T*)a.dt + s * a.dt_stride + c)));
        const T* bp = (const T*)a.B + s * a.b_stride + (int64_t)(c / per) * a.N;
        const T* cp = (const T*)a.Cm + s * a.c_stride + (int64_t)(c / per) * a.N;
        const float* Ap = a.A + (int64_t)c * a.N;
        const float xs = dt * x;
        float y = 0.f;
        if constexpr (VEC) {
            for (int n = 4 * q; n < a.N; n += 16) {
                f32x4 h = *(const f32x4*)(state + i * a.N + n);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(dt * (Ap[n + j] * kLog2e)), h[j],
                                          One<T>::widen(One<T>::load(bp + n + j)) * xs);
                    y = __builtin_fmaf(One<T>::widen(One<T>::load(cp + n + j)), h[j], y);
                }
                *(f32x4*)(state_out + i * a.N + n) = h;
            }
        } else {
            for (int n = q; n < a.N; n += 4) {
                const float h = __builtin_fmaf(__builtin_amdgcn_exp2f(dt * (Ap[n] * kLog2e)), state[i * a.N + n],
                                               One<T>::widen(One<T>::load(bp + n)) * xs);
                y = __builtin_fmaf(One<T>::widen(One<T>::load(cp + n)), h, y);
                state_out[i * a.N + n] = h;
            }
        }
        y += __shfl_xor(y, 1);
        y += __shfl_xor(y, 2);
        if (a.D) y += a.D[c] * x;
        if (a.z) {
            const float z = One<T>::widen(One<T>::load((const T*)a.z + s * a.z_stride + c));
            y *= z * sigmoid_f(z);
        }
        if (q == 0) store_one(a.y, i, a.y_f32, y);
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
        hipLaunchKernelGGL((selective_kernel<T, NS, true>), grid, block, 0, stream, a, lay, ends, steps);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int64_t blocks = ((int64_t)a.C * 4 * NS + 255) / 256 * a.nseq;
        hipLaunchKernelGGL(selective_carry_kernel, dim3((unsigned)std::min<int64_t>(blocks, kMaxBlocks)), dim3(256), 0,
                           stream, a, lay, ends, steps, 4 * NS);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((selective_kernel<T, NS, false>), grid, block, 0, stream, a, lay, ends, steps);
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
    const int64_t total = a.nseq * a.C;
    if (total == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>((total + 63) / 64, kMaxBlocks)), block(256);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, state, state_out); };
    const bool vec = a.N % 4 == 0;
    if (a.dtype == 1) vec ? go(selective_step_kernel<bf16_t, true>) : go(selective_step_kernel<bf16_t, false>);
    else vec ? go(selective_step_kernel<float, true>) : go(selective_step_kernel<float, false>);
    return hipGetLastError();
}

int64_t sel_saved_states(bool packed, int64_t nseq, int64_t L, int64_t T) {
    return sel_places(packed, nseq, L, T, kSelStateRows);
}

SelLayout sel_layout(const SelArgs& a, bool backward) {
    SelLayout l = {};
    const int64_t waves = (a.C + kSelChannels - 1) / kSelChannels, target = 4096;
    const int padded = a.N <= 4 ? 4 : a.N <= 8 ? 8 : a.N <= 16 ? 16 : a.N <= 32 ? 32 : 64;
    auto up = [](int64_t v) { return std::max<int64_t>((v + kSelStateRows - 1) / kSelStateRows, 1) * kSelStateRows; };
    if (!a.cu && a.nseq * waves >= target / 2) l.item = up(a.L);
    else l.item = up((int64_t)((double)a.T * waves / target));
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
