// Gated linear recurrence on gfx950: per sequence and channel, with gates
// computed from two logits of every token,
//   log a_t = -rate softplus(lam) sigmoid(r_t)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t,
// and its gradients.  A few dozen fp32 operations and 8 bytes (bf16) an
// element: an HBM stream, with the vector ALU close behind.
//
// The token axis of the whole batch is cut into tiles of kTileRows rows
// whatever the sequences' lengths; a sequence start inside a tile resets the
// state there.  A step is the map h -> a h + b, and a run of steps is again
// such a map (P, H): state at the end = P * (state before) + H.  A reset in a
// run makes P negative (its sign bit is the mark; P is never negative
// otherwise), so that nothing of the earlier sequence, NaN and infinities
// included, gets through a multiplication by 0.
//
// A decay near 1 is rounded to fp32 once (half of 2^-24); the factor P of a run
// comes from the sum of its log a, so these roundings do not add up from run
// to run over a memory of thousands of tokens.  1 - a^2 comes from a - 1, which
// is computed by itself.
#include <algorithm>

#include "ssd_gated.h"

namespace ssd {

namespace {

constexpr int kLaneCh = 4;                      // channels per lane
constexpr int kSegLanes = 16;                   // lanes across the channels of a row
constexpr int kTileCh = kLaneCh * kSegLanes;    // channels per workgroup
constexpr int kSegs = 16;                       // runs of rows per tile, one per 16 lanes
constexpr int kSegRows = 8;                     // rows per run
constexpr int kTileRows = kGatedTileRows;
static_assert(kSegs * kSegRows == kTileRows, "a tile is kSegs runs");
constexpr int kThreads = kSegs * kSegLanes;

__device__ inline bool is_reset(float P) { return __builtin_bit_cast(int, P) < 0; }

// The run after (P, H): applied to a state.
__device__ inline float advance(float P, float H, float h) { return is_reset(P) ? H : __builtin_fmaf(P, h, H); }

__device__ inline float nan_to_positive(float P) {
    return P != P ? __builtin_bit_cast(float, 0x7fc00000) : P;
}

// Boundary bits of the kSegRows rows from t0: bit j: row t0 + j is its
// sequence's first one; bit 16 + j: its last one.
__device__ inline uint32_t boundary_bits(const GatedArgs& a, int64_t t0) {
    uint32_t m = 0;
    if (!a.cu) {
        uint32_t p = (uint32_t)t0 % (uint32_t)a.L;  // rows < 2^31
        for (int64_t j = p ? a.L - p : 0; j <= kSegRows; j += a.L) {
            if (j < kSegRows) m |= 1u << j;
            if (j > 0) m |= 1u << (15 + j);
        }
        return m;
    }
    return a.bits[t0 / kSegRows];
}

// Packed batches: the boundary bits of every run of rows, and the states of
// sequences without tokens (their state passes through: out = in).
__global__ __launch_bounds__(256) void gated_plan_kernel(GatedArgs a, uint32_t* bits, const float* in, float* out) {
    const int64_t nruns = (a.T + kSegRows - 1) / kSegRows;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const RowRange live = live_rows(a.cu, a.nseq, a.T);
    for (int64_t k = me; bits && k < nruns; k += stride) {
        const int64_t t0 = k * kSegRows, t1 = min(t0 + kSegRows, live.hi);
        uint32_t m = 0;
        // every offset in [t0, t1] ends a sequence at the row before it and starts one at its row
        for (int64_t t = max(t0, live.lo); t <= t1;) {
            int64_t lo = 0, hi = a.nseq;  // the first offset >= t
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (a.cu[mid] < t) lo = mid + 1;
                else hi = mid;
            }
            const int64_t at = max((int64_t)a.cu[lo], t);
            if (at > t1) break;
            if (at < t1) m |= 1u << (at - t0);
            if (at > t0) m |= 1u << (15 + at - t0);
            t = at + 1;
        }
        bits[k] = m;
    }
    if (!out) return;
    const int64_t waves = stride / 64, lane = me & 63;
    for (int64_t s = me / 64; s < a.nseq; s += waves) {
        const RowRange q = seq_range(a.cu, a.L, a.T, s);
        if (q.hi > q.lo) continue;
        for (int64_t c = lane; c < a.C; c += 64) out[s * a.C + c] = in ? in[s * a.C + c] : 0.f;
    }
}

// What a lane has of its run of rows: the place, the boundary bits and the
// live rows (bit j).
struct Run {
    int64_t t0;
    int c0;          // first channel (clamped into the row)
    bool on;         // the lane's channels exist
    uint32_t bits, live;
    __device__ bool start(int j) const { return bits >> j & 1; }
    __device__ bool end(int j) const { return bits >> (16 + j) & 1; }
    __device__ bool has(int j) const { return live >> j & 1; }
};

__device__ inline Run this_run(const GatedArgs& a, int64_t tile, int cblock) {
    Run u;
    const int seg = threadIdx.x / kSegLanes;
    u.t0 = tile * kTileRows + seg * kSegRows;
    const int c = cblock * kTileCh + (threadIdx.x % kSegLanes) * kLaneCh;
    u.on = c < a.C;
    u.c0 = u.on ? c : a.C - kLaneCh;
    u.bits = u.t0 < a.T ? boundary_bits(a, u.t0) : 0;
    const RowRange r = live_rows(a.cu, a.nseq, a.T);
    const int lo = (int)min(max(r.lo - u.t0, (int64_t)0), (int64_t)kSegRows);
    const int hi = (int)min(max(r.hi - u.t0, (int64_t)lo), (int64_t)kSegRows);
    u.live = ((1u << hi) - 1) & ~((1u << lo) - 1);
    return u;
}

template <typename T>
__device__ inline void load_rows(const GatedArgs& a, const Run& u, const void* p, int64_t stride,
                                 typename Tr<T>::v4 (&v)[kSegRows]) {
#pragma unroll
    for (int j = 0; j < kSegRows; ++j)
        v[j] = Tr<T>::ld4raw((const T*)p + min(u.t0 + j, a.T - 1) * stride + u.c0);
}

// The factor of sigmoid(r) for the workgroup's channels, in LDS.
__device__ inline void load_factors(const GatedArgs& a, int cblock, float* k) {
    if (threadIdx.x < kTileCh)
        k[threadIdx.x] = decay_factor(a.lam[min(cblock * kTileCh + (int)threadIdx.x, a.C - 1)], a.rate);
}

__device__ inline f32x4 seq_state(const float* st, const GatedArgs& a, int64_t row, int c0) {
    return st ? *(const f32x4*)(st + seq_of(a.cu, a.nseq, a.L, row) * a.C + c0) : f32x4{};
}

// log a, the held decay and b of one row's four channels.
template <typename T>
struct Step {
    f32x4 loga, w, b;
    __device__ Step(f32x4 k, typename Tr<T>::v4 xv, typename Tr<T>::v4 rv, typename Tr<T>::v4 iv) {
        const f32x4 x = Tr<T>::widen4(xv), r = Tr<T>::widen4(rv), i = Tr<T>::widen4(iv);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            loga[c] = k[c] * sigmoid_f(r[c]);
            w[c] = held_decay(loga[c]);
            b[c] = __builtin_amdgcn_sqrtf(one_minus_a2(w[c])) * sigmoid_f(i[c]) * x[c];
        }
    }
    __device__ f32x4 a() const { return decay4(w); }
    __device__ static f32x4 decay4(f32x4 w) {
        return f32x4{decay_of(w[0]), decay_of(w[1]), decay_of(w[2]), decay_of(w[3])};
    }
};

// ------------------------------------------------------------------ forward
// The forward pass of one tile: with AGG only its map (P, H) per channel is
// written; otherwise the state entering the tile is read and y is written.
template <typename T, typename Y, bool AGG>
__global__ __launch_bounds__(kThreads) void gated_forward_kernel(GatedArgs a, f32x2* agg, const float* states) {
    __shared__ float k_s[kTileCh];
    __shared__ f32x4 P_s[kSegs][kSegLanes], H_s[kSegs][kSegLanes];
    const int seg = threadIdx.x / kSegLanes, ln = threadIdx.x % kSegLanes;
    const int64_t tile = blockIdx.x;
    const int cb = blockIdx.y;
    const Run u = this_run(a, tile, cb);
    load_factors(a, cb, k_s);
    typename Tr<T>::v4 xv[kSegRows], rv[kSegRows], iv[kSegRows];
    load_rows<T>(a, u, a.r, a.r_stride, rv);
    load_rows<T>(a, u, a.i, a.i_stride, iv);
    load_rows<T>(a, u, a.x, a.x_stride, xv);
    __syncthreads();
    const f32x4 k = *(const f32x4*)(k_s + ln * kLaneCh);

    f32x4 av[kSegRows], b[kSegRows], S = {}, H = {};
    bool reset = false;
#pragma unroll
    for (int j = 0; j < kSegRows; ++j) {
        const Step<T> st(k, xv[j], rv[j], iv[j]);
        av[j] = st.a();
        b[j] = st.b;
        if (u.has(j)) {
            if (u.start(j)) {
                H = seq_state(a.init, a, u.t0 + j, u.c0);
                reset = true;
            }
            S += st.loga;
            H = av[j] * H + b[j];
        }
    }
    f32x4 P;
#pragma unroll
    for (int c = 0; c < 4; ++c) P[c] = reset ? -1.f : nan_to_positive(__builtin_amdgcn_exp2f(S[c] * 1.44269504f));
    P_s[seg][ln] = P;
    H_s[seg][ln] = H;
    __syncthreads();
    // one lane per channel folds the runs
    if (threadIdx.x < kTileCh) {
        const int l = threadIdx.x / 4, c = threadIdx.x % 4, ch = cb * kTileCh + threadIdx.x;
        if constexpr (AGG) {
            float Pt = 1.f, Ht = 0.f;
            for (int s = 0; s < kSegs; ++s) {
                const float Pk = P_s[s][l][c];
                Ht = advance(Pk, H_s[s][l][c], Ht);
                Pt = is_reset(Pk) ? -1.f : Pt * Pk;
            }
            if (ch < a.C) agg[tile * a.C + ch] = f32x2{Pt, Ht};
        } else {
            float h = ch < a.C ? states[tile * a.C + ch] : 0.f;
            for (int s = 0; s < kSegs; ++s) {
                const float n = advance(P_s[s][l][c], H_s[s][l][c], h);
                H_s[s][l][c] = h;  // the state entering the run
                h = n;
            }
        }
    }
    if constexpr (!AGG) {
        __syncthreads();
        if (!u.on) return;
        f32x4 h = H_s[seg][ln];
#pragma unroll
        for (int j = 0; j < kSegRows; ++j) {
            if (!u.has(j)) continue;
            if (u.start(j)) h = seq_state(a.init, a, u.t0 + j, u.c0);
            h = av[j] * h + b[j];
            Tr<Y>::st4((Y*)a.y + (u.t0 + j) * a.C + u.c0, h);
            if (a.final_state && u.end(j))
                *(f32x4*)(a.final_state + seq_of(a.cu, a.nseq, a.L, u.t0 + j) * a.C + u.c0) = h;
        }
    }
}

// The state entering every tile, from the tiles' maps in order (REV: from the
// last one back: the adjoint entering every tile from behind).
template <bool REV>
__global__ __launch_bounds__(64) void gated_carry_kernel(int64_t ntiles, int C, const f32x2* agg, float* states) {
    const int ch = blockIdx.x * 64 + threadIdx.x;
    if (ch >= C) return;
    float h = 0.f;
    for (int64_t t = 0; t < ntiles; ++t) {
        const int64_t k = REV ? ntiles - 1 - t : t;
        states[k * C + ch] = h;
        const f32x2 m = agg[k * C + ch];
        h = advance(m[0], m[1], h);
    }
}

// ------------------------------------------------------------------ backward
// With q_{t+1} = a_{t+1} g_{t+1} the adjoint reaching token t from behind
// (dfinal at a sequence's last token): g_t = dy_t + q_{t+1}, and
//   dx = g beta sig(i),  di = g beta sig(i) (1 - sig(i)) x,
//   d log a = g (a h_{t-1} - a^2 / beta sig(i) x),
//   dr = dloga loga (1 - sig(r)),  dlam = sum dloga loga sigmoid(lam)/softplus(lam),
//   dinit = q at a sequence's first token.
// h_{t-1} is recomputed in fp32 from the state entering the tile.
template <typename T, typename Y, bool AGG>
__global__ __launch_bounds__(kThreads) void gated_backward_kernel(GatedArgs a, f32x2* agg, const float* adjoints,
                                                                  float* dlam_part) {
    __shared__ float k_s[kTileCh];
    __shared__ f32x4 P_s[kSegs][kSegLanes], H_s[kSegs][kSegLanes], R_s[kSegs][kSegLanes], Q_s[kSegs][kSegLanes];
    const int seg = threadIdx.x / kSegLanes, ln = threadIdx.x % kSegLanes;
    const int64_t tile = blockIdx.x;
    const int cb = blockIdx.y;
    const Run u = this_run(a, tile, cb);
    load_factors(a, cb, k_s);
    typename Tr<T>::v4 xv[kSegRows], rv[kSegRows], iv[kSegRows];
    typename Tr<Y>::v4 dv[kSegRows];
    load_rows<T>(a, u, a.r, a.r_stride, rv);
    load_rows<Y>(a, u, a.dy, a.C, dv);
    load_rows<T>(a, u, a.i, a.i_stride, iv);
    load_rows<T>(a, u, a.x, a.x_stride, xv);
    __syncthreads();
    const f32x4 k = *(const f32x4*)(k_s + ln * kLaneCh);

    f32x4 w[kSegRows], b[kSegRows], S = {}, H = {}, Q = {};
    bool reset = false, rreset = false;
#pragma unroll
    for (int j = 0; j < kSegRows; ++j) {
        const Step<T> st(k, xv[j], rv[j], iv[j]);
        w[j] = st.w;
        b[j] = st.b;
        if (u.has(j)) {
            if (u.start(j)) {
                H = seq_state(a.init, a, u.t0 + j, u.c0);
                reset = true;
            }
            rreset |= u.end(j);
            S += st.loga;
            H = st.a() * H + b[j];
        }
    }
#pragma unroll
    for (int j = kSegRows - 1; j >= 0; --j)
        if (u.has(j)) {
            if (u.end(j)) Q = seq_state(a.dfinal, a, u.t0 + j, u.c0);
            const f32x4 g = Q + Tr<Y>::widen4(dv[j]);
            Q = Step<T>::decay4(w[j]) * g;
        }
    f32x4 P;
#pragma unroll
    for (int c = 0; c < 4; ++c) P[c] = nan_to_positive(__builtin_amdgcn_exp2f(S[c] * 1.44269504f));
    const f32x4 marked = {-1.f, -1.f, -1.f, -1.f};
    P_s[seg][ln] = reset ? marked : P;
    H_s[seg][ln] = H;
    R_s[seg][ln] = rreset ? marked : P;
    Q_s[seg][ln] = Q;
    __syncthreads();
    if (threadIdx.x < kTileCh) {
        const int l = threadIdx.x / 4, c = threadIdx.x % 4, ch = cb * kTileCh + threadIdx.x;
        if constexpr (AGG) {
            float Pt = 1.f, Qt = 0.f;
            for (int s = kSegs - 1; s >= 0; --s) {
                const float Pk = R_s[s][l][c];
                Qt = advance(Pk, Q_s[s][l][c], Qt);
                Pt = is_reset(Pk) ? -1.f : Pt * Pk;
            }
            if (ch < a.C) agg[tile * a.C + ch] = f32x2{Pt, Qt};
        } else {
            float h = ch < a.C ? a.states_in[tile * a.C + ch] : 0.f, q = ch < a.C ? adjoints[tile * a.C + ch] : 0.f;
            for (int s = 0; s < kSegs; ++s) {
                const float n = advance(P_s[s][l][c], H_s[s][l][c], h);
                H_s[s][l][c] = h;
                h = n;
            }
            for (int s = kSegs - 1; s >= 0; --s) {
                const float n = advance(R_s[s][l][c], Q_s[s][l][c], q);
                Q_s[s][l][c] = q;
                q = n;
            }
        }
    }
    if constexpr (!AGG) {
        __syncthreads();
        f32x4 h = H_s[seg][ln], q = Q_s[seg][ln], before[kSegRows], dl = {};
#pragma unroll
        for (int j = 0; j < kSegRows; ++j)
            if (u.has(j)) {
                if (u.start(j)) h = seq_state(a.init, a, u.t0 + j, u.c0);
                before[j] = h;
                h = Step<T>::decay4(w[j]) * h + b[j];
            }
#pragma unroll
        for (int j = kSegRows - 1; j >= 0; --j) {
            if (!u.has(j)) continue;
            if (u.end(j)) q = seq_state(a.dfinal, a, u.t0 + j, u.c0);
            const f32x4 g = q + Tr<Y>::widen4(dv[j]);
            q = Step<T>::decay4(w[j]) * g;
            const f32x4 x = Tr<T>::widen4(xv[j]), r = Tr<T>::widen4(rv[j]), i = Tr<T>::widen4(iv[j]);
            f32x4 dx, di, dr;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float sr = sigmoid_f(r[c]), si = sigmoid_f(i[c]);
                // 1 - a^2 = 0 only where log a is 0, and its square root's reciprocal meets that factor below;
                // a floor (the least normal number) keeps their product 0 (a NaN passes)
                const float m0 = one_minus_a2(w[j][c]), m = m0 < 0x1p-126f ? 0x1p-126f : m0;
                const float rb = __builtin_amdgcn_rsqf(m), beta = m0 * rb, av = decay_of(w[j][c]);
                const float dl0 = g[c] * av * (before[j][c] - av * rb * si * x[c]) * (k[c] * sr);
                dx[c] = g[c] * beta * si;
                di[c] = dx[c] * x[c] * (1.f - si);
                dr[c] = dl0 * (1.f - sr);
                dl[c] += dl0;
            }
            if (!u.on) continue;
            Tr<T>::st4((T*)a.dx + (u.t0 + j) * a.dx_stride + u.c0, dx);
            Tr<T>::st4((T*)a.dr + (u.t0 + j) * a.dr_stride + u.c0, dr);
            Tr<T>::st4((T*)a.di + (u.t0 + j) * a.di_stride + u.c0, di);
            if (a.dinit && u.start(j))
                *(f32x4*)(a.dinit + seq_of(a.cu, a.nseq, a.L, u.t0 + j) * a.C + u.c0) = q;
        }
        __syncthreads();
        H_s[seg][ln] = dl;
        __syncthreads();
        if (threadIdx.x < kTileCh) {
            const int l = threadIdx.x / 4, c = threadIdx.x % 4, ch = cb * kTileCh + threadIdx.x;
            float s = 0.f;
            for (int j = 0; j < kSegs; ++j) s += H_s[j][l][c];
            if (ch < a.C) dlam_part[tile * a.C + ch] = s;
        }
    }
}

// dlam from the tiles' sums, in a fixed order: 16 lanes a channel take every
// 16th tile, then their sums are added.
__global__ __launch_bounds__(1024) void gated_dlam_kernel(GatedArgs a, int64_t ntiles, const float* part, float* dlam) {
    __shared__ float s_s[16][64];
    const int c = threadIdx.x & 63, strip = threadIdx.x >> 6, ch = blockIdx.x * 64 + c;
    float s = 0.f;
    if (ch < a.C)
        for (int64_t t = strip; t < ntiles; t += 16) s += part[t * a.C + ch];
    s_s[strip][c] = s;
    __syncthreads();
    if (strip || ch >= a.C) return;
    for (int j = 1; j < 16; ++j) s += s_s[j][c];
    // sigmoid(lam) / softplus(lam): 1 towards minus infinity, where both vanish
    const float lam = a.lam[ch], sp = softplus_f(lam);
    dlam[ch] = s * (sp < 1e-30f ? 1.f : (1.f / (1.f + expf(-lam))) / sp);
}

// ------------------------------------------------------------------ one token
template <typename T, typename Y>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedArgs a, const float* state, float* state_out) {
    const int64_t quads = a.C / kLaneCh;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.nseq * quads) return;
    const int64_t n = id / quads;
    const int c0 = (int)(id - n * quads) * kLaneCh;
    f32x4 h = *(const f32x4*)(state + n * a.C + c0), k = *(const f32x4*)(a.lam + c0);
    const Step<T> st((f32x4){decay_factor(k[0], a.rate), decay_factor(k[1], a.rate), decay_factor(k[2], a.rate),
                             decay_factor(k[3], a.rate)},
                     Tr<T>::ld4raw((const T*)a.x + n * a.x_stride + c0),
                     Tr<T>::ld4raw((const T*)a.r + n * a.r_stride + c0),
                     Tr<T>::ld4raw((const T*)a.i + n * a.i_stride + c0));
    h = st.a() * h + st.b;
    *(f32x4*)(state_out + n * a.C + c0) = h;
    Tr<Y>::st4((Y*)a.y + n * a.C + c0, h);
}

inline unsigned blocks_of(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

// The plan: boundary bits of a packed batch and the states of empty sequences.
hipError_t run_plan(const GatedArgs& a, uint32_t* bits, const float* in, float* out, hipStream_t stream) {
    if (!a.cu && a.T > 0) return hipSuccess;
    if (!bits && !out) return hipSuccess;
    const int64_t items = (a.T + kSegRows - 1) / kSegRows + a.nseq * 64;
    const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((items + 255) / 256, 1), 2048);
    hipLaunchKernelGGL(gated_plan_kernel, dim3(grid), dim3(256), 0, stream, a, bits, in, out);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_forward(GatedArgs a, const GatedLayout& lay, char* ws, hipStream_t stream) {
    uint32_t* bits = a.cu && a.T > 0 ? (uint32_t*)(ws + lay.bits) : nullptr;
    a.bits = bits;
    hipError_t e = run_plan(a, bits, a.init, a.final_state, stream);
    if (e != hipSuccess || a.T == 0) return e;
    float* states = a.states_out ? a.states_out : (float*)(ws + lay.carry);
    f32x2* agg = (f32x2*)(ws + lay.agg);
    const dim3 grid((unsigned)lay.ntiles, blocks_of(a.C, kTileCh));
    hipLaunchKernelGGL((gated_forward_kernel<T, Y, true>), grid, dim3(kThreads), 0, stream, a, agg, (const float*)nullptr);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((gated_carry_kernel<false>), dim3(blocks_of(a.C, 64)), dim3(64), 0, stream, lay.ntiles, a.C,
                       (const f32x2*)agg, states);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((gated_forward_kernel<T, Y, false>), grid, dim3(kThreads), 0, stream, a, agg, (const float*)states);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_backward(GatedArgs a, const GatedLayout& lay, char* ws, hipStream_t stream) {
    uint32_t* bits = a.cu && a.T > 0 ? (uint32_t*)(ws + lay.bits) : nullptr;
    a.bits = bits;
    hipError_t e = run_plan(a, bits, a.dfinal, a.dinit, stream);
    if (e != hipSuccess) return e;
    f32x2* agg = (f32x2*)(ws + lay.agg);
    float* adj = (float*)(ws + lay.carry);
    float* part = (float*)(ws + lay.dlam);
    if (a.T > 0) {
        const dim3 grid((unsigned)lay.ntiles, blocks_of(a.C, kTileCh));
        hipLaunchKernelGGL((gated_backward_kernel<T, Y, true>), grid, dim3(kThreads), 0, stream, a, agg,
                           (const float*)nullptr, (float*)nullptr);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((gated_carry_kernel<true>), dim3(blocks_of(a.C, 64)), dim3(64), 0, stream, lay.ntiles, a.C,
                           (const f32x2*)agg, adj);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((gated_backward_kernel<T, Y, false>), grid, dim3(kThreads), 0, stream, a, agg,
                           (const float*)adj, part);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(gated_dlam_kernel, dim3(blocks_of(a.C, 64)), dim3(1024), 0, stream, a, lay.ntiles,
                       (const float*)part, a.dlam);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_gated_step(const GatedArgs& a, const float* state, float* state_out, hipStream_t stream) {
    const int64_t n = a.nseq * (a.C / kLaneCh);
    if (n == 0) return hipSuccess;
    hipLaunchKernelGGL((gated_step_kernel<T, Y>), dim3(blocks_of(n, 256)), dim3(256), 0, stream, a, state, state_out);
    return hipGetLastError();
}

}  // namespace

GatedLayout gated_layout(int64_t T, int32_t C, bool packed, bool backward, bool keep_states) {
    GatedLayout l;
    l.ntiles = (T + kTileRows - 1) / kTileRows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    l.bits = take(packed ? (size_t)((T + kSegRows - 1) / kSegRows) * 4 : 0);
    l.agg = take((size_t)l.ntiles * C * 8);
    l.carry = take(backward || !keep_states ? (size_t)l.ntiles * C * 4 : 0);
    l.dlam = take(backward ? (size_t)l.ntiles * C * 4 : 0);
    l.total = at;
    return l;
}

hipError_t launch_gated_scan(const GatedArgs& a, const GatedLayout& lay, void* ws, hipStream_t stream) {
    char* w = (char*)ws;
    if (a.dtype == 1)
        return a.y_f32 ? run_forward<bf16_t, float>(a, lay, w, stream) : run_forward<bf16_t, bf16_t>(a, lay, w, stream);
    return a.y_f32 ? run_forward<float, float>(a, lay, w, stream) : run_forward<float, bf16_t>(a, lay, w, stream);
}

hipError_t launch_gated_backward(const GatedArgs& a, const GatedLayout& lay, void* ws, hipStream_t stream) {
    char* w = (char*)ws;
    if (a.dtype == 1)
        return a.y_f32 ? run_backward<bf16_t, float>(a, lay, w, stream) : run_backward<bf16_t, bf16_t>(a, lay, w, stream);
    return a.y_f32 ? run_backward<float, float>(a, lay, w, stream) : run_backward<float, bf16_t>(a, lay, w, stream);
}

hipError_t launch_gated_step(const GatedArgs& a, const float* state, float* state_out, hipStream_t stream) {
    if (a.dtype == 1)
        return a.y_f32 ? run_gated_step<bf16_t, float>(a, state, state_out, stream)
                       : run_gated_step<bf16_t, bf16_t>(a, state, state_out, stream);
    return a.y_f32 ? run_gated_step<float, float>(a, state, state_out, stream)
                   : run_gated_step<float, bf16_t>(a, state, state_out, stream);
}

}  // namespace ssd
