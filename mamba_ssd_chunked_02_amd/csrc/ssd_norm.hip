// RMS norms around a block on gfx950, each fused with the elementwise work
// that touches the same rows:
//   residual norm   out = residual + scale x,   y = out rstd w
//   gated norm      v = x silu(z),              y = v rstd w
//                   (or y = x rstd w silu(z): the norm before the gate)
// with rstd = 1 / sqrt(mean(v^2) + eps) per row, or per group of a row.
// A few operations per element read: HBM streams.  A row is held in
// registers between the sum and its use, so every input is read once.
//
// A row of up to 4096 columns is one wave's (no LDS, no barrier: the four
// waves of a workgroup run apart), a longer one a workgroup's.  A lane takes
// 8 consecutive columns at a time.
#include <algorithm>

#include "ssd_column_sum.h"
#include "ssd_device.h"

namespace ssd {

namespace {

constexpr int kNormThreads = 256;
constexpr int kVec = 8;

__device__ inline float sigm(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

// Sum over the lanes that share a row (WPR waves), the same in every lane.
template <int WPR>
__device__ inline float row_sum(float v, float* lds) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if constexpr (WPR > 1) {
        __syncthreads();  // the last sum's readers are done
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += lds[w];
    }
    return v;
}

template <int WPR>
struct Place {
    static constexpr int kLanes = 64 * WPR;
    int lane;
    __device__ Place() : lane(WPR == 1 ? threadIdx.x & 63 : threadIdx.x) {}
    __device__ int col(int v) const { return (v * kLanes + lane) * kVec; }
};

__device__ inline float sum8(f32x8 v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// silu(z) and its derivative.
__device__ inline f32x8 silu8(f32x8 z) {
    f32x8 g;
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = z[e] * sigm(z[e]);
    return g;
}

// ------------------------------------------------------------------ forward
// KIND 0: residual norm (A: type of x and y, B: of the residual).
// KIND 1: gated norm (A: type of z and y, B: of x); 2: the norm before the gate.
template <typename A, typename B, int KIND, int WPR, int V>
__global__ __launch_bounds__(kNormThreads) void norm_forward_kernel(NormArgs a) {
    __shared__ float lds[4];
    const Place<WPR> p;
    const int64_t seg = WPR == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
    if (seg >= a.rows * a.G) return;  // WPR 1: whole waves; else: whole workgroups
    const int64_t row = seg / a.G;
    const int n = a.D / a.G, g0 = (int)(seg - row * a.G) * n;
    const A* xa = KIND == 0 ? (const A*)a.x + row * a.x_stride + g0 : (const A*)a.z + row * a.z_stride + g0;
    const B* xb = KIND == 0 ? (const B*)a.z + row * a.z_stride + g0 : (const B*)a.x + row * a.x_stride + g0;
    f32x8 u[V], gate[V];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = p.col(v);
        u[v] = f32x8{};
        if (c < n) {
            const f32x8 va = Tr<A>::widen(Tr<A>::ld8(xa + c));
            const f32x8 vb = Tr<B>::widen(Tr<B>::ld8(xb + c));
            if constexpr (KIND == 0) {
                u[v] = a.scale ? vb + Tr<float>::ld8(a.scale + g0 + c) * va : vb + va;
                Tr<B>::st8((B*)a.out + row * a.D + g0 + c, Tr<B>::narrow(u[v]));
            } else {
                gate[v] = silu8(va);
                u[v] = KIND == 1 ? vb * gate[v] : vb;
            }
            ss += sum8(u[v] * u[v]);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<WPR>(ss, lds) / (float)n + a.eps);
    if (a.rstd && p.lane == 0) a.rstd[seg] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = p.col(v);
        if (c < n) {
            f32x8 y = u[v] * rstd * Tr<float>::ld8(a.weight + g0 + c);
            if constexpr (KIND == 2) y *= gate[v];
            Tr<A>::st8((A*)a.y + row * a.D + g0 + c, Tr<A>::narrow(y));
        }
    }
}

// ------------------------------------------------------------------ backward
// With m = v rstd the normalised row and d the gradient of m w:
//   dv = rstd (w d - m mean(w d m)),  dw = sum over rows of d m.
// A workgroup takes every gridDim.x-th row (set of four rows) and keeps its
// sums of dw (and dscale) in registers; they go to its own row of the partial
// sums, which a second kernel adds in a fixed order.
template <typename A, typename B, int KIND, int WPR, int V>
__global__ __launch_bounds__(kNormThreads) void norm_backward_kernel(NormArgs a) {
    __shared__ float lds[4];
    __shared__ f32x4 sums[WPR == 1 ? 3 * 64 * V * 2 : 1];
    const Place<WPR> p;
    const int n = a.D / a.G, g0 = blockIdx.y * n;
    constexpr int kRows = WPR == 1 ? 4 : 1;
    const int wave = WPR == 1 ? threadIdx.x >> 6 : 0;
    const bool scaled = KIND == 0 && a.dscale;
    f32x8 w[V], dw[V] = {}, ds[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = p.col(v) < n ? Tr<float>::ld8(a.weight + g0 + p.col(v)) : f32x8{};
    for (int64_t row = (int64_t)blockIdx.x * kRows + wave; row < a.rows; row += (int64_t)gridDim.x * kRows) {
        const float rstd = a.rstd_in[row * a.G + blockIdx.y];
        f32x8 m[V], wd[V], vx[V], vz[V];
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = p.col(v);
            m[v] = wd[v] = vx[v] = vz[v] = f32x8{};
            if (c < n) {
                const f32x8 dy = Tr<A>::widen(Tr<A>::ld8((const A*)a.dy + row * a.D + g0 + c));
                if constexpr (KIND == 0) {
                    m[v] = Tr<B>::widen(Tr<B>::ld8((const B*)a.out + row * a.D + g0 + c)) * rstd;
                    wd[v] = dy * w[v];
                    dw[v] += dy * m[v];
                } else {
                    vx[v] = Tr<B>::widen(Tr<B>::ld8((const B*)a.x + row * a.x_stride + g0 + c));
                    vz[v] = Tr<A>::widen(Tr<A>::ld8((const A*)a.z + row * a.z_stride + g0 + c));
                    const f32x8 gate = silu8(vz[v]);
                    m[v] = (KIND == 1 ? vx[v] * gate : vx[v]) * rstd;
                    const f32x8 d = KIND == 1 ? dy : dy * gate;
                    wd[v] = d * w[v];
                    dw[v] += d * m[v];
                    if constexpr (KIND == 2) vx[v] = dy;  // x itself is no longer needed
                }
                dot += sum8(wd[v] * m[v]);
            }
        }
        const float mean = row_sum<WPR>(dot, lds) / (float)n;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = p.col(v);
            if (c >= n) continue;
            f32x8 dv = (wd[v] - m[v] * mean) * rstd;
            if constexpr (KIND == 0) {
                if (a.dout) dv += Tr<B>::widen(Tr<B>::ld8((const B*)a.dout + row * a.D + g0 + c));
                if (a.dz) Tr<B>::st8((B*)a.dz + row * a.D + g0 + c, Tr<B>::narrow(dv));
                if (scaled) ds[v] += dv * Tr<A>::widen(Tr<A>::ld8((const A*)a.x + row * a.x_stride + g0 + c));
                if (a.dx) {
                    if (a.scale) dv *= Tr<float>::ld8(a.scale + g0 + c);
                    Tr<A>::st8((A*)a.dx + row * a.D + g0 + c, Tr<A>::narrow(dv));
                }
            } else {
                f32x8 dx, dz;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = vz[v][e], s = sigm(z), dsilu = s * (1.f + z * (1.f - s));
                    if (KIND == 1) {
                        dx[e] = dv[e] * (z * s);
                        dz[e] = dv[e] * vx[v][e] * dsilu;
                    } else {
                        dx[e] = dv[e];
                        dz[e] = vx[v][e] * w[v][e] * m[v][e] * dsilu;
                    }
                }
                Tr<B>::st8((B*)a.dx + row * a.dx_stride + g0 + c, Tr<B>::narrow(dx));
                Tr<A>::st8((A*)a.dz + row * a.dz_stride + g0 + c, Tr<A>::narrow(dz));
            }
        }
    }
    // this workgroup's sums over its rows
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && !scaled) break;
        f32x8(&s)[V] = k ? ds : dw;
        float* to = a.part + ((int64_t)k * a.nparts + blockIdx.x) * a.D + g0;
        if constexpr (WPR == 1) {
            __syncthreads();
            if (wave) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sums[(((wave - 1) * V + v) * 2) * 64 + p.lane] = __builtin_shufflevector(s[v], s[v], 0, 1, 2, 3);
                    sums[(((wave - 1) * V + v) * 2 + 1) * 64 + p.lane] = __builtin_shufflevector(s[v], s[v], 4, 5, 6, 7);
                }
            }
            __syncthreads();
            if (wave) continue;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int o = 0; o < 3; ++o) {
                    const f32x4 lo = sums[((o * V + v) * 2) * 64 + p.lane], hi = sums[((o * V + v) * 2 + 1) * 64 + p.lane];
                    s[v] += __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (p.col(v) < n) Tr<float>::st8(to + p.col(v), s[v]);
    }
}

__global__ __launch_bounds__(kSumThreads) void column_sum_kernel(const float* part, int64_t n, int64_t ld, int cols,
                                                                 float* out) {
    const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const float s = column_sum(n, [&](int64_t t) { return col < cols ? part[t * ld + col] : 0.f; });
    if (threadIdx.x < kSumCols && col < cols) out[col] = s;
}

template <typename A, typename B, int KIND, int WPR, int V>
hipError_t run_norm(const NormArgs& a, bool backward, hipStream_t stream) {
    if (backward) {
        if (a.rows > 0) {
            hipLaunchKernelGGL((norm_backward_kernel<A, B, KIND, WPR, V>), dim3(a.nparts, a.G), dim3(kNormThreads), 0,
                               stream, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        const hipError_t e = launch_column_sum(a.part, a.rows > 0 ? a.nparts : 0, a.D, a.D, a.dweight, stream);
        if (e != hipSuccess || !a.dscale) return e;
        return launch_column_sum(a.part + (int64_t)a.nparts * a.D, a.rows > 0 ? a.nparts : 0, a.D, a.D, a.dscale, stream);
    }
    const int64_t segs = a.rows * a.G, blocks = WPR == 1 ? (segs + 3) / 4 : segs;
    if (segs == 0) return hipSuccess;
    hipLaunchKernelGGL((norm_forward_kernel<A, B, KIND, WPR, V>), dim3((unsigned)blocks), dim3(kNormThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename A, typename B, int KIND>
hipError_t by_columns(const NormArgs& a, bool backward, hipStream_t stream) {
    const int n = a.D / a.G;
    if (n <= 4096) switch ((n + 511) / 512) {
            case 1: return run_norm<A, B, KIND, 1, 1>(a, backward, stream);
            case 2: return run_norm<A, B, KIND, 1, 2>(a, backward, stream);
            case 3: return run_norm<A, B, KIND, 1, 3>(a, backward, stream);
            case 4: return run_norm<A, B, KIND, 1, 4>(a, backward, stream);
            case 5: return run_norm<A, B, KIND, 1, 5>(a, backward, stream);
            case 6: return run_norm<A, B, KIND, 1, 6>(a, backward, stream);
            default: return run_norm<A, B, KIND, 1, 8>(a, backward, stream);
        }
    switch ((n + 2047) / 2048) {
        case 3: return run_norm<A, B, KIND, 4, 3>(a, backward, stream);
        case 4: return run_norm<A, B, KIND, 4, 4>(a, backward, stream);
        case 5:
        case 6: return run_norm<A, B, KIND, 4, 6>(a, backward, stream);
        case 7:
        case 8: return run_norm<A, B, KIND, 4, 8>(a, backward, stream);
        default: return hipErrorInvalidValue;
    }
}

// The two types: a_f32 that of x and y (residual norm) or z and y (gated
// norm), b_f32 that of the residual or x; fp32 with a bf16 second is refused.
template <int KIND>
hipError_t by_types(const NormArgs& a, bool backward, hipStream_t stream) {
    if (a.a_f32) return a.b_f32 ? by_columns<float, float, KIND>(a, backward, stream) : hipErrorInvalidValue;
    return a.b_f32 ? by_columns<bf16_t, float, KIND>(a, backward, stream)
                   : by_columns<bf16_t, bf16_t, KIND>(a, backward, stream);
}

}  // namespace

int32_t norm_parts(int64_t rows, int32_t D, int32_t G) {
    const int64_t per = D / G <= 4096 ? 4 : 1;  // rows a workgroup works on at once
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, std::max(1, 1024 / G)));
}

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t stream) { return by_types<0>(a, false, stream); }
hipError_t launch_residual_norm_backward(const NormArgs& a, hipStream_t stream) { return by_types<0>(a, true, stream); }
hipError_t launch_gated_norm(const NormArgs& a, hipStream_t stream) {
    return a.norm_first ? by_types<2>(a, false, stream) : by_types<1>(a, false, stream);
}
hipError_t launch_gated_norm_backward(const NormArgs& a, hipStream_t stream) {
    return a.norm_first ? by_types<2>(a, true, stream) : by_types<1>(a, true, stream);
}

hipError_t launch_column_sum(const float* part, int64_t n, int64_t ld, int32_t cols, float* out, hipStream_t stream) {
    hipLaunchKernelGGL(column_sum_kernel, dim3((cols + kSumCols - 1) / kSumCols), dim3(kSumThreads), 0, stream, part, n, ld, cols, out);
    return hipGetLastError();
}

}  // namespace ssd
