// Layer norm on gfx950, with the residual addition of the block before:
//   u = residual + scale x   (or u = x),   y = (u - mean(u)) rstd w + b
// with rstd = 1 / sqrt(mean((u - mean(u))^2) + eps) per row.
// A few operations per element read: HBM streams.  A row is held in registers
// between its sums and its use, so every input is read once.  65536 x 2560, bf16 with
// an fp32 residual: forward 334 us, backward 481 (6.0 and 5.6 TB/s), with a scale 527 (5.7);
// 16384 x 5120, bf16: 77 and 102 us (4.4 and 4.9).
//
// The mean is taken first and the squares of the distances from it then, both from
// registers: a row whose mean is large against its spread keeps its digits.  The
// first mean's own rounding shows in the sum of the distances, which comes with the
// second sum, and is taken off again.
#include <type_traits>

#include "ssd_norm_rows.h"

namespace ssd {

namespace {

constexpr int64_t kMaxBlocks = 1 << 22;  // a launch counts its lanes in 32 bits
constexpr int kBackWaves = 10;           // of a workgroup of the backward pass

// Vectors of 8 columns a lane of the backward pass: one up to 8 waves a row (10 with a
// residual), else as few as 8 waves allow.  16384 x 5120, bf16: two vectors 102 us, one 144.
inline int backward_vectors(int n, int kind) {
    return n <= (kind == kNormPlain ? 8 : kBackWaves) * 64 * kVec ? 1 : norm_vectors(n);
}

// ------------------------------------------------------------------ forward
// A: type of x and y, B: of the residual (RES).
template <typename A, typename B, bool RES, int LANES, bool WIDE, int V>
__global__ __launch_bounds__(WIDE ? 64 * kMaxWaves : 256) void layer_norm_kernel(NormArgs a) {
    __shared__ float lds[kMaxWaves], lds2[kMaxWaves][2];
    constexpr bool SPLIT = sizeof(A) == 4 || (RES && sizeof(B) == 4);
    typedef Eight<A, SPLIT> EA;
    typedef Eight<B, SPLIT> EB;
    typedef Eight<float, SPLIT> EW;
    const Team<LANES, WIDE, V> p;
    const int n = a.D;
    // as many rounds as the workgroup's first team has: a team without a row
    // still takes part in its wave's shuffles
    const int64_t first = (int64_t)blockIdx.x * (WIDE ? 1 : (int)blockDim.x / LANES);
    for (int64_t s0 = first, row = p.index; s0 < a.rows; s0 += p.teams, row += p.teams) {
        const bool on = row < a.rows;
        const int64_t at = on ? row * n : 0;
        typename EA::raw ra[V];
        typename EB::raw rb[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, on ? n : 0);
            ra[v] = EA::load((const A*)a.x + at, k);
            if constexpr (RES) rb[v] = EB::load((const B*)a.z + at, k);
        }
        f32x8 u[V];
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, on ? n : 0);
            u[v] = EA::widen(ra[v]);
            if constexpr (RES) {
                const f32x8 r = EB::widen(rb[v]);
                u[v] = a.scale ? r + EW::cached(a.scale, k) * u[v] : r + u[v];
                EB::store((B*)a.out + at, k, u[v]);
            }
            sum += sum8(u[v]);
        }
        const float mean = p.sum(sum, lds) / (float)n;
        float rest = 0.f, ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, on ? n : 0);
            u[v] = away_from(u[v], mean, k);
            rest += sum8(u[v]);
            ss += sum8(u[v] * u[v]);
        }
        p.sum2(rest, ss, lds2);
        rest /= (float)n;
        // NaN stays NaN; squares that overflow leave rstd at 0, also where the mean's rounding does so, too
        const float var = ss / (float)n - fminf(rest * rest, 3.4028234e38f);
        const float rstd = 1.f / sqrtf(__builtin_elementwise_maximum(var, 0.f) + a.eps);
        if (!on) continue;
        if (p.lane == 0) {
            if (a.mean) a.mean[row] = fabsf(mean) < __builtin_inff() ? mean + rest : mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, n);
            f32x8 y = (u[v] - rest) * rstd * EW::cached(a.weight, k);
            if (a.bias) y += EW::cached(a.bias, k);
            EA::store((A*)a.y + at, k, y);
        }
    }
}

// ------------------------------------------------------------------ backward
// With m = (u - mean) rstd and d the gradient of y:
//   du = dout + rstd (w d - mean(w d) - m mean(w d m)),  dx = scale du,
//   dw = sum over rows of d m,  db of d,  dscale of du x.
// Team k takes the rows k, k + teams, ..., mostly with the next one's data in flight, and keeps
// its sums over rows in registers; a workgroup's go to its own row of the partial
// sums, which a second kernel adds.

// Waves of a SIMD, and so registers a lane and workgroups at once.  With a residual
// three, since the compiler at four waits for its loads early (65536 x 2560 bf16: 281
// us, four 347; with an fp32 residual 480, 519), and with a scale none of the next row's
// (527; with them 685, four waves without them 610).  fp32 without a residual: three
// for one vector a lane (65536 x 1024: 138, four 149), four for two (16384 x 5120: 176
// with 3 of them in scratch, three 208); bf16 four (16384 x 4096: 83, three 108; 16384 x 8192 147, three with the next row 180).
// Four vectors a lane, over 8192 columns, do not fit with a residual: 11 to 19 registers go
// to scratch (8192 x 12288 bf16 246 us, 4.1 TB/s), with a scale 74 to 100 (513 us, 2.4).
constexpr int backward_waves(int kind, bool f32, int V) {
    return kind == kNormPlain && V <= 2 ? (V == 1 && f32 ? 3 : 4) : V == 1 ? 3 : 2;
}

// KIND: kNormResidual, there may be a gradient of the sum and a second output; kNormScaled, a scale too.
template <typename A, typename B, int KIND, int LANES, bool WIDE, int V>
__global__ __launch_bounds__(!WIDE ? 256 : V == 1 ? 64 * kBackWaves : 64 * kMaxWaves,
                             backward_waves(KIND, sizeof(A) == 4, V)) void layer_norm_backward_kernel(NormArgs a) {
    __shared__ float lds[kBackWaves][2];
    __shared__ f32x4 sums[WIDE ? 1 : 3 * 64 * V * 2];
    constexpr bool SPLIT = sizeof(A) == 4 || sizeof(B) == 4;
    typedef Eight<A, SPLIT> EA;
    typedef Eight<B, SPLIT> EB;
    typedef Eight<float, SPLIT> EW;
    const Team<LANES, WIDE, V> p;
    const int n = a.D;
    const bool scaled = KIND == kNormScaled && a.dscale;
    struct Row {
        typename EA::raw dy[V], x[V];
        typename EB::raw u[V], dout[V];
        float mean, rstd;
    };
    auto load = [&](int64_t row, Row& r) {
        const bool there = row < a.rows;
        r.mean = there ? a.mean_in[row] : 0.f;
        r.rstd = there ? a.rstd_in[row] : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, there ? n : 0);
            r.dy[v] = EA::load((const A*)a.dy + row * n, k);
            r.u[v] = EB::load((const B*)a.out + row * n, k);
            if constexpr (KIND == kNormPlain) continue;
            r.dout[v] = {};
            r.x[v] = {};
            if (a.dout) r.dout[v] = EB::load((const B*)a.dout + row * n, k);
            if (scaled) r.x[v] = EA::load((const A*)a.x + row * n, k);
        }
    };
    f32x8 w[V], dw[V] = {}, db[V] = {}, ds[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols k = p.template cols<SPLIT>(v, n);
        w[v] = EW::cached(a.weight, k);
    }
    constexpr bool kAhead = V == 1 ? KIND != kNormScaled : V == 2 && KIND == kNormResidual;  // the next row's loads
    Row cur, nxt;
    if (kAhead) load(p.index, nxt);
    // WIDE: the same rows for the whole workgroup; else as many rounds as the
    // workgroup's first team has, so that a wave's teams stay together
    const int64_t first = (int64_t)blockIdx.x * (WIDE ? 1 : (int)blockDim.x / LANES);
    for (int64_t r0 = first, row = p.index; r0 < a.rows; r0 += p.teams, row += p.teams) {
        if (kAhead) {
            cur = nxt;
            load(row + p.teams, nxt);
        } else {
            load(row, cur);
        }
        f32x8 m[V], wd[V];
        float mean1 = 0.f, mean2 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const f32x8 d = EA::widen(cur.dy[v]);
            m[v] = (EB::widen(cur.u[v]) - cur.mean) * cur.rstd;
            wd[v] = d * w[v];
            dw[v] += d * m[v];
            db[v] += d;
            mean1 += sum8(wd[v]);
            mean2 += sum8(wd[v] * m[v]);
        }
        p.sum2(mean1, mean2, lds);
        mean1 /= (float)n;
        mean2 /= (float)n;
        if (row >= a.rows) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, n);
            f32x8 du = (wd[v] - mean1 - m[v] * mean2) * cur.rstd;
            if constexpr (KIND != kNormPlain) {
                du += EB::widen(cur.dout[v]);
                if (a.dz) EB::store((B*)a.dz + row * n, k, du);
                if (scaled) ds[v] += du * EA::widen(cur.x[v]);
                if constexpr (KIND == kNormScaled) du *= EW::cached(a.scale, k);  // read again: registers are short
            }
            EA::store((A*)a.dx + row * n, k, du);
        }
    }
    // this workgroup's sums over its rows
    auto out = [&](f32x8(&s)[V], int o) {
        float* to = a.part + ((int64_t)o * a.nparts + blockIdx.x) * n;
        if constexpr (!WIDE) {
            // the wave's teams hold the same columns; then waves 1..3 through LDS
#pragma unroll
            for (int d = LANES; d < 64; d <<= 1)
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[v][e] += __shfl_xor(s[v][e], d);
            const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
            __syncthreads();
            if (wave) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sums[(((wave - 1) * V + v) * 2) * 64 + lane] = __builtin_shufflevector(s[v], s[v], 0, 1, 2, 3);
                    sums[(((wave - 1) * V + v) * 2 + 1) * 64 + lane] = __builtin_shufflevector(s[v], s[v], 4, 5, 6, 7);
                }
            }
            __syncthreads();
            if (wave || lane >= LANES) return;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const f32x4 lo = sums[((i * V + v) * 2) * 64 + lane], hi = sums[((i * V + v) * 2 + 1) * 64 + lane];
                    s[v] += __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) EW::store_cached(to, p.template cols<SPLIT>(v, n), s[v]);
    };
    out(dw, 0);
    if (a.dbias) out(db, 1);
    if (scaled) out(ds, 2);
}

// dweight, dbias and dscale (blockIdx.y: which of those wanted) from the workgroups' partial sums.
__global__ __launch_bounds__(kSumThreads) void layer_norm_sums_kernel(NormArgs a, int64_t n) {
    float* const to[3] = {a.dweight, a.dbias, a.dscale};
    const int o = blockIdx.y == 0 ? 0 : blockIdx.y == 1 && a.dbias ? 1 : 2;
    const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const float* part = a.part + (int64_t)o * a.nparts * a.D;
    const float s = column_sum(n, [&](int64_t t) { return col < a.D ? part[t * a.D + col] : 0.f; });
    if (threadIdx.x < kSumCols && col < a.D) to[o][col] = s;
}

template <typename A, typename B, bool RES, int LANES, bool WIDE, int V>
hipError_t run_forward(const NormArgs& a, hipStream_t stream) {
    const int threads = WIDE ? norm_threads(a.D, V) : 256, per = WIDE ? 1 : 256 / LANES;
    if (a.rows == 0) return hipSuccess;
    const int64_t blocks = std::min<int64_t>((a.rows + per - 1) / per, kMaxBlocks);
    hipLaunchKernelGGL((layer_norm_kernel<A, B, RES, LANES, WIDE, V>), dim3((unsigned)blocks), dim3(threads), 0, stream, a);
    return hipGetLastError();
}

template <typename A, typename B, int KIND, int LANES, bool WIDE, int V>
hipError_t run_backward(const NormArgs& a, hipStream_t stream) {
    if (a.rows > 0) {
        hipLaunchKernelGGL((layer_norm_backward_kernel<A, B, KIND, LANES, WIDE, V>), dim3(a.nparts),
                           dim3(WIDE ? norm_threads(a.D, V) : 256), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(layer_norm_sums_kernel,
                       dim3((a.D + kSumCols - 1) / kSumCols, 1 + (a.dbias != nullptr) + (a.dscale != nullptr)),
                       dim3(kSumThreads), 0, stream, a, (int64_t)(a.rows > 0 ? a.nparts : 0));
    return hipGetLastError();
}

// Forward, rows of 513 to 2560 columns go to one wave each, which needs no barrier for
// its two sums (65536 x 1536, bf16: 83 us, over a workgroup's waves 102; 32768 x 2560,
// fp32: 113, 128); wider ones to two to four waves (16384 x 5120, bf16: two waves 77 us, one 83, five 87).
template <typename A, typename B, bool RES>
hipError_t forward_by_columns(const NormArgs& a, hipStream_t stream) {
    const int n = a.D;
    if (n <= 8 * kVec) return run_forward<A, B, RES, 8, false, 1>(a, stream);
    if (n <= 16 * kVec) return run_forward<A, B, RES, 16, false, 1>(a, stream);
    if (n <= 32 * kVec) return run_forward<A, B, RES, 32, false, 1>(a, stream);
    if (n <= 64 * kVec) return run_forward<A, B, RES, 64, false, 1>(a, stream);
    if (n <= 2 * 64 * kVec) return run_forward<A, B, RES, 64, false, 2>(a, stream);
    if (n <= 3 * 64 * kVec) return run_forward<A, B, RES, 64, false, 3>(a, stream);
    if (n <= 5 * 64 * kVec) return run_forward<A, B, RES, 64, false, 5>(a, stream);
    if (n <= 8 * 64 * kVec) return run_forward<A, B, RES, 64, true, 4>(a, stream);
    if (n <= 10 * 64 * kVec) return run_forward<A, B, RES, 64, true, 5>(a, stream);
    return run_forward<A, B, RES, 64, true, 4>(a, stream);
}

template <typename A, typename B, int KIND>
hipError_t backward_by_columns(const NormArgs& a, hipStream_t stream) {
    const int n = a.D;
    if (n <= 8 * kVec) return run_backward<A, B, KIND, 8, false, 1>(a, stream);
    if (n <= 16 * kVec) return run_backward<A, B, KIND, 16, false, 1>(a, stream);
    if (n <= 32 * kVec) return run_backward<A, B, KIND, 32, false, 1>(a, stream);
    if (n <= 64 * kVec) return run_backward<A, B, KIND, 64, false, 1>(a, stream);
    switch (backward_vectors(n, KIND)) {
        case 1: return run_backward<A, B, KIND, 64, true, 1>(a, stream);
        case 2: return run_backward<A, B, KIND, 64, true, 2>(a, stream);
        default: return run_backward<A, B, KIND, 64, true, 4>(a, stream);
    }
}

}  // namespace

// Workgroups along the rows of the backward pass: what 256 compute units hold at once,
// no more than there are rows for.  By registers 16 waves are three workgroups of 5 waves,
// but a third one does not start beside two: of 768 over 5120 columns 256 started when the
// others ended.  Hence a power of two of each compute unit: 65536 x 5120 without a residual
// 2 332 us, 3 399, fp32 676 and 748.  Where they all start at once it is quicker, too, for a
// reason not known: 65536 x 1024 with an fp32 residual 4 186 us, 6 206, fp32 137 and 144; but
// not for bf16 rows without a residual by one vector, which have the least in flight and
// take all of them: 65536 x 2560 3 184 us, 2 227; x 1536 5 111, 4 120.  The quicker side
// is the same one for 12000, 16384, 20011, 24000, 32768 and 50000 rows.
int32_t layer_norm_parts(int64_t rows, int32_t D, int kind, bool f32) {
    const int V = backward_vectors(D, kind), narrow = D <= 8 * kVec ? 8 : D <= 16 * kVec ? 16 : D <= 32 * kVec ? 32 : 64;
    const bool wide = D > 64 * kVec;
    const int per = wide ? 1 : 256 / narrow, waves = wide ? norm_threads(D, V) / 64 : 4;
    int held = std::max(1, 4 * backward_waves(kind, f32, V) / waves);
    while ((held & (held - 1)) && (kind != kNormPlain || f32 || V > 1)) held &= held - 1;
    held *= 256;
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, held));
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t stream) {
    if (!a.z)
        return a.a_f32 ? forward_by_columns<float, float, false>(a, stream)
                       : forward_by_columns<bf16_t, bf16_t, false>(a, stream);
    if (a.a_f32) return forward_by_columns<float, float, true>(a, stream);
    return a.b_f32 ? forward_by_columns<bf16_t, float, true>(a, stream)
                   : forward_by_columns<bf16_t, bf16_t, true>(a, stream);
}

int layer_norm_kind(const NormArgs& a) {
    return a.scale ? kNormScaled : a.dout || a.dz || a.a_f32 != a.b_f32 ? kNormResidual : kNormPlain;
}

hipError_t launch_layer_norm_backward(const NormArgs& a, hipStream_t stream) {
    const int kind = layer_norm_kind(a);
    if (a.a_f32)
        return kind == kNormPlain      ? backward_by_columns<float, float, kNormPlain>(a, stream)
               : kind == kNormResidual ? backward_by_columns<float, float, kNormResidual>(a, stream)
                                   : backward_by_columns<float, float, kNormScaled>(a, stream);
    if (a.b_f32)
        return kind == kNormResidual ? backward_by_columns<bf16_t, float, kNormResidual>(a, stream)
                                 : backward_by_columns<bf16_t, float, kNormScaled>(a, stream);
    return kind == kNormPlain      ? backward_by_columns<bf16_t, bf16_t, kNormPlain>(a, stream)
           : kind == kNormResidual ? backward_by_columns<bf16_t, bf16_t, kNormResidual>(a, stream)
                               : backward_by_columns<bf16_t, bf16_t, kNormScaled>(a, stream);
}

}  // namespace ssd
