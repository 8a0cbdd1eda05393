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
// (every 64 tokens): first those entering every 16 tokens, which a lane keeps in
// LDS, then a tile's, which it keeps in registers with the decays.
#include <algorithm>
#include <type_traits>

#include "ssd_column_sum.h"
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kWaves = kSelBackChannels / kSelChannels;  // of a workgroup
constexpr int kSub = 16;   // tokens between two states in LDS
constexpr int kSubs = (int)kSelStateRows / kSub;
constexpr int64_t kMaxBlocks = 1 << 22;
constexpr float kLn2 = 0.693147180559945309f;

// ---------------------------------------------------------------- sums over channels
// Lane k of a row: the sum of v[k] over the row's 16 lanes.  Every step sends half
// of what a lane holds to the lane opposite.
template <int CTRL>
__device__ inline float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ inline float sum_channels(const float (&v)[16], int k) {
    float a[8], b[4], c[2];
    const bool b3 = k & 8, b2 = k & 4, b1 = k & 2, b0 = k & 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (b3 ? v[i + 8] : v[i]) + dpp<0x140>(b3 ? v[i] : v[i + 8]);  // row_mirror
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = (b2 ? a[i + 4] : a[i]) + dpp<0x141>(b2 ? a[i] : a[i + 4]);  // row_half_mirror
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = (b1 ? b[i + 2] : b[i]) + dpp<0x1b>(b1 ? b[i] : b[i + 2]);   // quad_perm:[3,2,1,0]
    return (b0 ? c[1] : c[0]) + dpp<0xb1>(b0 ? c[0] : c[1]);                                       // quad_perm:[1,0,3,2]
}

template <typename T, int NS>
__device__ inline void load_states_of(const T* p, int64_t stride, int t0, int n, int N, int q, int k,
                                      typename One<T>::raw (&to)[SelTile<NS>::NB]) {
#pragma unroll
    for (int i = 0; i < SelTile<NS>::NB; ++i) {
        const int f = 16 * i + k, s = min(q * NS + f % NS, N - 1);
        to[i] = One<T>::load(p + (int64_t)min(t0 + f / NS, n - 1) * stride + s);
    }
}
template <typename T, int NS>
__device__ inline void widen_states_of(const typename One<T>::raw (&r)[SelTile<NS>::NB], int t0, int n, int N, int q,
                                       int k, float (&to)[SelTile<NS>::NB]) {
#pragma unroll
    for (int i = 0; i < SelTile<NS>::NB; ++i) {
        const int f = 16 * i + k;
        to[i] = q * NS + f % NS < N && t0 + f / NS < n ? One<T>::widen(r[i]) : 0.f;
    }
}
// dy is of y's type, which may not be x's.
template <typename T>
__device__ inline float load_dy(const SelArgs& a, int64_t at) {
    return a.y_f32 ? ((const float*)a.dy)[at] : One<bf16_t>::widen(One<bf16_t>::load((const bf16_t*)a.dy + at));
}

// ---------------------------------------------------------------- adjoints of items, from zero
// The gradient that an item hands to the token before it if none enters at its end,
// for all items but a sequence's first.
template <typename T, int NS>
__global__ __launch_bounds__(256) void selective_adjoint_kernel(SelArgs a, SelLayout lay, float* ends, float* steps) {
    typedef SelTile<NS> G;
    constexpr int TT = G::TT, Q = G::Q;
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = a.C / a.G, nblk = (per + 4 * kSelChannels - 1) / (4 * kSelChannels) * a.G;
    const int64_t work = lay.places * nblk;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / (nblk / a.G);
        const SelItem e = sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place);
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
            A[j] = s < a.N ? a.A[(int64_t)c * a.N + s] * kLog2e : 0.f;
            ga[j] = 0.f;
        }
        const StepSize step(a.act, c);
        float total = 0.f;
        const T* dp = (const T*)a.dt + e.lo * a.dt_stride + c;
        const T* zp = (const T*)a.z + e.lo * a.z_stride + c;
        const T* cp = (const T*)a.Cm + e.lo * a.c_stride + g * a.N;
        for (int t0 = (n - 1) / TT * TT; t0 >= 0; t0 -= TT) {
            typename One<T>::raw rc[G::NB];
            float cc[G::NB];
            load_states_of<T, NS>(cp, a.c_stride, t0, n, a.N, q, k, rc);
            widen_states_of<T, NS>(rc, t0, n, a.N, q, k, cc);
            unroll<Q>([&](auto group) {
                constexpr int i = Q - 1 - decltype(group)::value;
                if (t0 + 4 * i >= n) return;
                const int t = t0 + 4 * i + q;
                const bool there = t < n;
                const int64_t row = min(t, n - 1);
                const float dt = there ? step(One<T>::widen(One<T>::load(dp + row * a.dt_stride))) : 0.f;
                float u = load_dy<T>(a, (e.lo + row) * a.C + c);
                if (a.z) {
                    const float z = One<T>::widen(One<T>::load(zp + row * a.z_stride));
                    u *= z * sigmoid_f(z);
                }
                total += dt;
                float dts[4], us[4];
                rows_to_all(dt, dts);
                rows_to_all(there ? u : 0.f, us);
                unroll<4>([&](auto token) {
                    constexpr int t = 3 - decltype(token)::value;
                    if (t0 + 4 * i + t >= n) return;
                    unroll<NS>([&](auto state) {
                        constexpr int j = decltype(state)::value, f = (4 * i + t) * NS + j;
                        ga[j] = __builtin_amdgcn_exp2f(dts[t] * A[j]) *
                                __builtin_fmaf(row_lane<f % 16>(cc[f / 16]), us[t], ga[j]);
                    });
                });
            });
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
        const float A = there ? a.A[(int64_t)c * a.N + n] * kLog2e : 0.f;
        float h = a.dfinal && there ? a.dfinal[(s * a.C + c) * a.N + n] : 0.f;
        const int64_t place = sel_place(a.cu != nullptr, s, r.lo, a.L, lay.item) + items - 1;
        float* p = ends + place * row + at;
        const float* st = steps + place * a.C + c;
        for (int64_t j = items - 1; j > 0; --j, p -= row, st -= a.C) {
            h = __builtin_fmaf(__builtin_amdgcn_exp2f(A * *st), h, *p);
            *p = h;
        }
    }
}

// ---------------------------------------------------------------- gradients
template <typename T, int NS>
__global__ __launch_bounds__(64 * kWaves) void selective_backward_kernel(SelArgs a, SelLayout lay, const float* ends,
                                                                         float* part_bc, float* part_a) {
    typedef SelTile<NS> G;
    constexpr int TT = G::TT, NB = G::NB, Q = G::Q;
    __shared__ float s_h[kWaves][kSubs][NS][64];
    __shared__ float s_bc[2][kWaves][2][NB][64];
    const int lane = threadIdx.x & 63, q = lane >> 4, k = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per = a.C / a.G, gblk = (int)lay.blocks_bc, nblk = gblk * a.G;
    const int64_t work = lay.places * nblk;
    int buf = 0;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int64_t place = w / nblk;
        const int cb = (int)(w - place * nblk), g = cb / gblk, block = cb - g * gblk;
        const SelItem e = sel_item(a.cu, a.nseq, a.L, a.T, lay.item, place);
        const int c0 = g * per + (block * kWaves + wave) * kSelChannels, end = (g + 1) * per;
        const bool on = c0 + k < end;
        const int c = on ? c0 + k : end - 1;  // lanes without a channel: gradients of zero
        const int n = e.seq < 0 ? 0 : (int)e.n;
        const int64_t chan = (int64_t)c * a.N;

        float A[NS], ga[NS], dA[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            const int s = q * NS + j;
            A[j] = s < a.N ? a.A[chan + s] * kLog2e : 0.f;
            dA[j] = ga[j] = 0.f;
            if (e.seq < 0 || !on) continue;
            if (!e.last) ga[j] = ends[((place + 1) * a.C + c) * (4 * NS) + s];
            else if (a.dfinal && s < a.N) ga[j] = a.dfinal[e.seq * a.C * a.N + chan + s];
        }
        const StepSize step(a.act, c);
        const float D = a.D ? a.D[c] : 0.f;
        float dD = 0.f, dbias = 0.f;

        const T* xp = (const T*)a.x + e.lo * a.x_stride + c;
        const T* dp = (const T*)a.dt + e.lo * a.dt_stride + c;
        const T* zp = (const T*)a.z + e.lo * a.z_stride + c;
        const T* bp = (const T*)a.B + e.lo * a.b_stride + g * a.N;
        const T* cp = (const T*)a.Cm + e.lo * a.c_stride + g * a.N;

        float h[NS];
        // the states over the TT tokens from t0, which are all there
        auto advance = [&](int t0) {
            typename One<T>::raw rb[NB];
            float b[NB];
            load_states_of<T, NS>(bp, a.b_stride, t0, n, a.N, q, k, rb);
            widen_states_of<T, NS>(rb, t0, n, a.N, q, k, b);
            unroll<Q>([&](auto group) {
                constexpr int i = decltype(group)::value;
                const int64_t row = t0 + 4 * i + q;
                const float dt = step(One<T>::widen(One<T>::load(dp + row * a.dt_stride)));
                const float x = One<T>::widen(One<T>::load(xp + row * a.x_stride));
                float dts[4], xs[4];
                rows_to_all(dt, dts);
                rows_to_all(on ? dt * x : 0.f, xs);
                unroll<4>([&](auto token) {
                    constexpr int t = decltype(token)::value;
                    unroll<NS>([&](auto state) {
                        constexpr int j = decltype(state)::value, f = (4 * i + t) * NS + j;
                        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(dts[t] * A[j]), h[j],
                                              row_lane<f % 16>(b[f / 16]) * xs[t]);
                    });
                });
            });
        };
        // gradients of the tile of t0, h the state entering it
        auto tile = [&](int t0, auto tail) {
            constexpr bool TAIL = decltype(tail)::value;
            typename One<T>::raw rb[NB], rc[NB];
            float b[NB], cc[NB], x[Q], raw[Q], dt[Q], dy[Q], z[Q], u[Q];
            load_states_of<T, NS>(bp, a.b_stride, t0, n, a.N, q, k, rb);
            load_states_of<T, NS>(cp, a.c_stride, t0, n, a.N, q, k, rc);
            widen_states_of<T, NS>(rb, t0, n, a.N, q, k, b);
            widen_states_of<T, NS>(rc, t0, n, a.N, q, k, cc);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int64_t row = min(t0 + 4 * i + q, n - 1);
                const bool there = on && (!TAIL || t0 + 4 * i + q < n);
                x[i] = there ? One<T>::widen(One<T>::load(xp + row * a.x_stride)) : 0.f;
                raw[i] = One<T>::widen(One<T>::load(dp + row * a.dt_stride));
                dt[i] = there ? step(raw[i]) : 0.f;
                u[i] = dy[i] = there ? load_dy<T>(a, (e.lo + row) * a.C + c) : 0.f;
                z[i] = 0.f;
                if (a.z) {
                    z[i] = there ? One<T>::widen(One<T>::load(zp + row * a.z_stride)) : 0.f;
                    u[i] = dy[i] * (z[i] * sigmoid_f(z[i]));
                }
            }
            float before[TT][NS], decay[TT][NS], last[NS];
            unroll<Q>([&](auto group) {
                constexpr int i = decltype(group)::value;
                float dts[4], xs[4];
                rows_to_all(dt[i], dts);
                rows_to_all(dt[i] * x[i], xs);
                unroll<4>([&](auto token) {
                    constexpr int t = decltype(token)::value;
                    unroll<NS>([&](auto state) {
                        constexpr int j = decltype(state)::value, f = (4 * i + t) * NS + j;
                        before[4 * i + t][j] = h[j];
                        decay[4 * i + t][j] = 1.f;
                        if (TAIL && t0 + 4 * i + t >= n) return;
                        decay[4 * i + t][j] = __builtin_amdgcn_exp2f(dts[t] * A[j]);
                        h[j] = __builtin_fmaf(decay[4 * i + t][j], h[j], row_lane<f % 16>(b[f / 16]) * xs[t]);
                    });
                });
            });
#pragma unroll
            for (int j = 0; j < NS; ++j) last[j] = h[j];
            float pb[NB][16], pc[NB][16];
            unroll<Q>([&](auto group) {
                constexpr int i = Q - 1 - decltype(group)::value;
                float dts[4], xs[4], us[4], s[4], ew[4], y[4];
                rows_to_all(dt[i], dts);
                rows_to_all(dt[i] * x[i], xs);
                rows_to_all(u[i], us);
                unroll<4>([&](auto token) {
                    constexpr int t = 3 - decltype(token)::value, at = 4 * i + t;
                    s[t] = ew[t] = y[t] = 0.f;
                    if (TAIL && t0 + at >= n) {
                        unroll<NS>([&](auto state) {
                            constexpr int f = at * NS + decltype(state)::value;
                            pb[f / 16][f % 16] = pc[f / 16][f % 16] = 0.f;
                        });
                        return;
                    }
                    unroll<NS>([&](auto state) {
                        constexpr int j = decltype(state)::value, f = at * NS + j;
                        const float C = row_lane<f % 16>(cc[f / 16]);
                        const float now = at + 1 < TT ? before[at + 1 < TT ? at + 1 : 0][j] : last[j];
                        const float adj = __builtin_fmaf(us[t], C, ga[j]);
                        pc[f / 16][f % 16] = us[t] * now;
                        pb[f / 16][f % 16] = adj * xs[t];
                        y[t] = __builtin_fmaf(C, now, y[t]);
                        s[t] = __builtin_fmaf(row_lane<f % 16>(b[f / 16]), adj, s[t]);
                        ga[j] = adj * decay[at][j];
                        const float wn = ga[j] * before[at][j];
                        ew[t] = __builtin_fmaf(wn, A[j], ew[t]);
                        dA[j] = __builtin_fmaf(wn, dts[t], dA[j]);
                    });
                });
                const float S = sum_rows(s), E = sum_rows(ew) * kLn2;
                const float Y = a.z ? sum_rows(y) + D * x[i] : 0.f;
                const bool there = on && (!TAIL || t0 + 4 * i + q < n);
                if (there) {
                    const int64_t row = e.lo + t0 + 4 * i + q;
                    const float draw = (x[i] * S + E) * step.slope(raw[i], dt[i]);
                    const bool f32 = std::is_same<T, float>::value;
                    store_one(a.dx, row * a.dx_stride + c, f32, dt[i] * S + D * u[i]);
                    store_one(a.ddt, row * a.ddt_stride + c, f32, draw);
                    dbias += draw;
                    dD += u[i] * x[i];
                    if (a.z) {
                        const float sg = sigmoid_f(z[i]);
                        store_one(a.dz, row * a.dz_stride + c, f32, dy[i] * Y * (sg * (1.f + z[i] * (1.f - sg))));
                    }
                }
            });
            // the workgroup's sums over its channels
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                s_bc[buf][wave][0][i][lane] = sum_channels(pb[i], k);
                s_bc[buf][wave][1][i][lane] = sum_channels(pc[i], k);
            }
            __syncthreads();
            for (int o = threadIdx.x; o < 2 * NB * 64; o += 64 * kWaves) {
                const int l = o & 63, i = (o >> 6) % NB, which = (o >> 6) / NB;
                const int f = 16 * i + (l & 15), s = (l >> 4) * NS + f % NS, t = t0 + f / NS;
                if (t >= n || s >= a.N) continue;
                float v = 0.f;
#pragma unroll
                for (int o2 = 0; o2 < kWaves; ++o2) v += s_bc[buf][o2][which][i][l];
                part_bc[(((int64_t)block * a.T + e.lo + t) * a.G + g) * (2 * a.N) + which * a.N + s] = v;
            }
            buf ^= 1;  // the readers of this one are done before the barrier after the next
        };
        for (int chunk = n > 0 ? (n - 1) / (int)kSelStateRows * (int)kSelStateRows : -1; chunk >= 0;
             chunk -= (int)kSelStateRows) {
            const int64_t slot = sel_place(a.cu != nullptr, e.seq, e.first, a.L, kSelStateRows) +
                                 (e.index * lay.item + chunk) / kSelStateRows;
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const int s = q * NS + j;
                h[j] = on && s < a.N ? a.states_in[slot * a.C * a.N + chan + s] : 0.f;
            }
            const int subs = (min(n - chunk, (int)kSelStateRows) + kSub - 1) / kSub;
            for (int sub = 0; sub < subs; ++sub) {
                if (sub)
                    for (int t = 0; t < kSub; t += TT) advance(chunk + (sub - 1) * kSub + t);
#pragma unroll
                for (int j = 0; j < NS; ++j) s_h[wave][sub][j][lane] = h[j];
            }
            for (int sub = subs - 1; sub >= 0; --sub) {
                const int base = chunk + sub * kSub, here = min(n - base, kSub);
                for (int t = (here - 1) / TT * TT; t >= 0; t -= TT) {
#pragma unroll
                    for (int j = 0; j < NS; ++j) h[j] = s_h[wave][sub][j][lane];
                    for (int o = 0; o < t; o += TT) advance(base + o);
                    if (t + TT <= here) tile(base + t, std::false_type{});
                    else tile(base + t, std::true_type{});
                }
            }
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
    const int64_t width = (int64_t)a.C * (a.N + 2);
    const int64_t col = (int64_t)blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const float v = column_sum(places, [&](int64_t t) { return col < width ? part[t * width + col] : 0.f; });
    if (threadIdx.x >= kSumCols || col >= width) return;
    const int64_t states = (int64_t)a.C * a.N;
    if (col < states) a.dA[col] = v;
    else if (col < states + a.C) {
        if (a.dD) a.dD[col - states] = v;
    } else if (a.dbias) a.dbias[col - states - a.C] = v;
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
        hipLaunchKernelGGL((selective_backward_kernel<T, NS>), dim3((unsigned)std::min<int64_t>(work, kMaxBlocks)),
                           dim3(64 * kWaves), 0, stream, a, lay, ends, part_bc, part_a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if (a.T > 0) {
            const int64_t elements = a.T * a.G * 2 * a.N;
            hipLaunchKernelGGL((selective_sum_bc_kernel<T>),
                               dim3((unsigned)std::min<int64_t>((elements + 255) / 256, 1 << 16)), dim3(256), 0, stream,
                               a, part_bc, lay.blocks_bc);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    const int64_t columns = (int64_t)a.C * (a.N + 2);
    hipLaunchKernelGGL(selective_sum_kernel, dim3((unsigned)((columns + kSumCols - 1) / kSumCols)), dim3(kSumThreads), 0,
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
