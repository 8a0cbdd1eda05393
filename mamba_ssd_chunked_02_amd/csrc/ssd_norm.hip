// RMS norms around a block on gfx950, each fused with the elementwise work
// that touches the same rows:
//   residual norm   out = residual + scale x,   y = out rstd w
//   gated norm      v = x silu(z),              y = v rstd w
//                   (or y = x rstd w silu(z): the norm before the gate)
// with rstd = 1 / sqrt(mean(v^2) + eps) per row, or per group of a row.
// A few operations per element read: HBM streams.  A row is held in
// registers between the sum and its use, so every input is read once.
//
// A row (or group of a row) belongs to a team of lanes, 8 columns each at a time:
// 8 to 64 lanes of a wave, or all waves of a workgroup where it is wider.
// Wide rows over many waves with few registers a lane beat one wave with many
// (65536 rows of 2560 columns, forward and backward: 5 waves a row and the
// next row in flight 974 us, one wave a row 1069 us; 256 rows forward 4.2
// against 5.8 us), and narrow groups share a wave.  Now: those rows, with an
// fp32 residual, 916 us, 5.5 TB/s; 49152 rows of 8192 columns in 8 groups,
// gated, forward and backward 1160 us, 5.5 TB/s.
#include <algorithm>
#include <type_traits>

#include "ssd_column_sum.h"
#include "ssd_device.h"

namespace ssd {

namespace {

constexpr int kVec = 8;
constexpr int kMaxWaves = 8;
constexpr int64_t kMaxBlocks = 1 << 22;  // a launch counts its lanes in 32 bits

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A lane's 8 columns are consecutive, 16 bytes of bf16 and whole lines a wave,
// which stream past the caches (the data is read and written once; 49152 rows of
// 8192 columns forward and backward 1159 us, cached 1180 us).  fp32 takes two
// accesses that share every line, and so needs the cache between them.  SPLIT,
// the residual norm where a type is fp32: two times 4 consecutive columns, half
// a team's width apart, so that fp32 too is streamed in whole lines (65536 rows of
// 2560 columns with an fp32 residual 921 us, consecutive and cached 967 us).  The
// gated norm keeps to consecutive columns: with one fp32 tensor in five halves
// lose (358 against 350 us for 16384 rows of 5120); with fp32 x and z they would
// win forward (161 against 184 us there, 264 against 303 us for 8192 rows of 16384)
// and win or lose 2 or 3% backward (308 against 314 us, 725 against 706 us).
struct Cols {
    int c[2];
    bool on[2];
};

template <typename T, bool SPLIT>
struct Eight;
template <bool SPLIT>
struct Eight<bf16_t, SPLIT> {
    typedef u32x4 raw;
    __device__ static inline raw load(const bf16_t* p, const Cols& k) {
        raw r = {};
        if constexpr (!SPLIT) {
            if (k.on[0]) r = __builtin_nontemporal_load((const raw*)(p + k.c[0]));
        } else {
            u32x2 lo = {}, hi = {};
            if (k.on[0]) lo = __builtin_nontemporal_load((const u32x2*)(p + k.c[0]));
            if (k.on[1]) hi = __builtin_nontemporal_load((const u32x2*)(p + k.c[1]));
            r = raw{lo[0], lo[1], hi[0], hi[1]};
        }
        return r;
    }
    __device__ static inline f32x8 widen(raw v) {
        f32x8 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[2 * e] = __builtin_bit_cast(float, v[e] << 16);
            r[2 * e + 1] = __builtin_bit_cast(float, v[e] & 0xffff0000u);
        }
        return r;
    }
    __device__ static inline void store(bf16_t* p, const Cols& k, f32x8 v) {
        const bf16x8 n = Tr<bf16_t>::narrow(v);
        if constexpr (!SPLIT) {
            if (k.on[0]) __builtin_nontemporal_store(n, (bf16x8*)(p + k.c[0]));
        } else {
            if (k.on[0]) __builtin_nontemporal_store(__builtin_shufflevector(n, n, 0, 1, 2, 3), (bf16x4*)(p + k.c[0]));
            if (k.on[1]) __builtin_nontemporal_store(__builtin_shufflevector(n, n, 4, 5, 6, 7), (bf16x4*)(p + k.c[1]));
        }
    }
};
template <bool SPLIT>
struct Eight<float, SPLIT> {
    typedef f32x8 raw;
    __device__ static inline const float* second(const float* p, const Cols& k) { return p + (SPLIT ? k.c[1] : k.c[0] + 4); }
    __device__ static inline bool has_second(const Cols& k) { return k.on[SPLIT ? 1 : 0]; }
    __device__ static inline raw load(const float* p, const Cols& k) {
        if constexpr (!SPLIT) return cached(p, k);
        f32x4 lo = {}, hi = {};
        if (k.on[0]) lo = __builtin_nontemporal_load((const f32x4*)(p + k.c[0]));
        if (k.on[1]) hi = __builtin_nontemporal_load((const f32x4*)(p + k.c[1]));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // weights, and what is summed over rows
    __device__ static inline raw cached(const float* p, const Cols& k) {
        f32x4 lo = {}, hi = {};
        if (k.on[0]) lo = *(const f32x4*)(p + k.c[0]);
        if (has_second(k)) hi = *(const f32x4*)second(p, k);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ static inline f32x8 widen(raw v) { return v; }
    __device__ static inline void store(float* p, const Cols& k, f32x8 v) {
        if constexpr (!SPLIT) return store_cached(p, k, v);
        if (k.on[0]) __builtin_nontemporal_store(__builtin_shufflevector(v, v, 0, 1, 2, 3), (f32x4*)(p + k.c[0]));
        if (k.on[1]) __builtin_nontemporal_store(__builtin_shufflevector(v, v, 4, 5, 6, 7), (f32x4*)(p + k.c[1]));
    }
    __device__ static inline void store_cached(float* p, const Cols& k, f32x8 v) {
        if (k.on[0]) *(f32x4*)(p + k.c[0]) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
        if (has_second(k)) *(f32x4*)second(p, k) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    }
};

__device__ inline float sigm(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}
__device__ inline float sum8(f32x8 v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
__device__ inline f32x8 silu8(f32x8 z) {
    f32x8 g;
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = z[e] * sigm(z[e]);
    return g;
}

// LANES < 64: a team is LANES lanes of a wave.  64: a wave, or (WIDE) all
// waves of the workgroup.
template <int LANES, bool WIDE, int V>
struct Team {
    int lane, stride;  // lane of the team; columns from one of the lane's vectors to the next
    int64_t index, teams;
    __device__ Team() {
        const int per = WIDE ? 1 : (int)blockDim.x / LANES;
        lane = WIDE ? (int)threadIdx.x : (int)threadIdx.x % LANES;
        stride = (WIDE ? (int)blockDim.x : LANES) * kVec;
        index = (int64_t)blockIdx.x * per + (WIDE ? 0 : (int)threadIdx.x / LANES);
        teams = (int64_t)gridDim.x * per;
    }
    // The lane's columns of its v-th vector, and whether a row of n columns has them.
    template <bool SPLIT>
    __device__ Cols cols(int v, int n) const {
        Cols k;
        k.c[0] = v * stride + lane * (SPLIT ? 4 : kVec);
        k.c[1] = k.c[0] + (SPLIT ? stride / 2 : 0);
        k.on[0] = k.c[0] < n;
        k.on[1] = k.c[1] < n;
        return k;
    }
    // Sum over the team, the same in every lane.
    __device__ float sum(float v, float* lds) const {
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) v += __shfl_xor(v, d);
        if constexpr (WIDE) {
            __syncthreads();  // the last sum's readers are done
            if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
            __syncthreads();
            v = 0.f;
            for (int w = 0; w < (int)blockDim.x / 64; ++w) v += lds[w];
        }
        return v;
    }
};

// ------------------------------------------------------------------ forward
// KIND 0: residual norm (A: type of x and y, B: of the residual).
// KIND 1: gated norm (A: type of z and y, B: of x); 2: the norm before the gate.
template <typename A, typename B, int KIND, int LANES, bool WIDE, int V>
__global__ __launch_bounds__(WIDE ? 64 * kMaxWaves : 256) void norm_forward_kernel(NormArgs a) {
    __shared__ float lds[kMaxWaves];
    constexpr bool SPLIT = KIND == 0 && (sizeof(A) == 4 || sizeof(B) == 4);
    typedef Eight<A, SPLIT> EA;
    typedef Eight<B, SPLIT> EB;
    typedef Eight<float, SPLIT> EW;
    const Team<LANES, WIDE, V> p;
    const int n = a.D / a.G;
    const int64_t segs = a.rows * a.G;
    // as many rounds as the workgroup's first team has: a team without a row
    // still takes part in its wave's shuffles
    const int64_t first = (int64_t)blockIdx.x * (WIDE ? 1 : (int)blockDim.x / LANES);
    for (int64_t s0 = first, seg = p.index; s0 < segs; s0 += p.teams, seg += p.teams) {
        const bool on = seg < segs;
        const int64_t row = on ? seg / a.G : 0;
        const int g0 = on ? (int)(seg - row * a.G) * n : 0;
        const A* xa = KIND == 0 ? (const A*)a.x + row * a.x_stride + g0 : (const A*)a.z + row * a.z_stride + g0;
        const B* xb = KIND == 0 ? (const B*)a.z + row * a.z_stride + g0 : (const B*)a.x + row * a.x_stride + g0;
        typename EA::raw ra[V];
        typename EB::raw rb[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, on ? n : 0);
            ra[v] = EA::load(xa, k);
            rb[v] = EB::load(xb, k);
        }
        f32x8 u[V], gate[V];
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, on ? n : 0);
            const f32x8 va = EA::widen(ra[v]), vb = EB::widen(rb[v]);
            if constexpr (KIND == 0) {
                u[v] = a.scale ? vb + EW::cached(a.scale + g0, k) * va : vb + va;
                EB::store((B*)a.out + row * a.D + g0, k, u[v]);
            } else {
                gate[v] = silu8(va);
                u[v] = KIND == 1 ? vb * gate[v] : vb;
            }
            ss += sum8(u[v] * u[v]);
        }
        const float rstd = 1.f / sqrtf(p.sum(ss, lds) / (float)n + a.eps);
        if (!on) continue;
        if (a.rstd && p.lane == 0) a.rstd[seg] = rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, n);
            f32x8 y = u[v] * rstd * EW::cached(a.weight + g0, k);
            if constexpr (KIND == 2) y *= gate[v];
            EA::store((A*)a.y + row * a.D + g0, k, y);
        }
    }
}

// ------------------------------------------------------------------ backward
// With m = v rstd the normalised row and d the gradient of m w:
//   dv = rstd (w d - m mean(w d m)),  dw = sum over rows of d m.
// Team k takes the rows k, k + teams, ..., the next one's data in flight, and
// keeps its sums of dw (and dscale) in registers; a workgroup's go to its own row
// of the partial sums, which a second kernel adds.
template <typename A, typename B, int KIND, int LANES, bool WIDE, int V>
__global__ __launch_bounds__(WIDE ? 64 * kMaxWaves : 256, V == 1 ? 4 : 2) void norm_backward_kernel(NormArgs a) {
    __shared__ float lds[kMaxWaves];
    __shared__ f32x4 sums[WIDE ? 1 : 3 * 64 * V * 2];
    constexpr bool SPLIT = KIND == 0 && (sizeof(A) == 4 || sizeof(B) == 4);
    typedef Eight<A, SPLIT> EA;
    typedef Eight<B, SPLIT> EB;
    typedef Eight<float, SPLIT> EW;
    const Team<LANES, WIDE, V> p;
    const int n = a.D / a.G, g0 = blockIdx.y * n;
    const bool scaled = KIND == 0 && a.dscale;
    // KIND 0: dy, the new residual, its gradient, x;  else: dy, x, z
    struct Row {
        typename EA::raw dy[V], za[V];
        typename EB::raw xb[V], db[V];
        float rstd;
    };
    auto load = [&](int64_t row, Row& r) {
        const bool there = row < a.rows;
        r.rstd = there ? a.rstd_in[row * a.G + blockIdx.y] : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, there ? n : 0);
            const int64_t dense = row * a.D + g0;
            r.dy[v] = EA::load((const A*)a.dy + dense, k);
            if constexpr (KIND == 0) {
                r.xb[v] = EB::load((const B*)a.out + dense, k);
                r.za[v] = {};
                r.db[v] = {};
                if (a.dout) r.db[v] = EB::load((const B*)a.dout + dense, k);
                if (scaled) r.za[v] = EA::load((const A*)a.x + row * a.x_stride + g0, k);
            } else {
                r.xb[v] = EB::load((const B*)a.x + row * a.x_stride + g0, k);
                r.za[v] = EA::load((const A*)a.z + row * a.z_stride + g0, k);
            }
        }
    };
    f32x8 w[V], sc[V], dw[V] = {}, ds[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Cols k = p.template cols<SPLIT>(v, n);
        w[v] = EW::cached(a.weight + g0, k);
        if (KIND == 0) sc[v] = a.scale ? EW::cached(a.scale + g0, k) : f32x8{1, 1, 1, 1, 1, 1, 1, 1};
    }
    constexpr bool kAhead = V < 4;  // there are no registers for the next row of the widest ones
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
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f32x8 d = EA::widen(cur.dy[v]);
            const f32x8 xb = EB::widen(cur.xb[v]);
            if constexpr (KIND == 0) {
                m[v] = xb * cur.rstd;
            } else {
                const f32x8 gate = silu8(EA::widen(cur.za[v]));
                m[v] = (KIND == 1 ? xb * gate : xb) * cur.rstd;
                if (KIND == 2) d *= gate;
            }
            wd[v] = d * w[v];
            dw[v] += d * m[v];
            dot += sum8(wd[v] * m[v]);
        }
        const float mean = p.sum(dot, lds) / (float)n;
        if (row >= a.rows) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Cols k = p.template cols<SPLIT>(v, n);
            f32x8 dv = (wd[v] - m[v] * mean) * cur.rstd;
            if constexpr (KIND == 0) {
                dv += EB::widen(cur.db[v]);
                const int64_t dense = row * a.D + g0;
                if (a.dz) EB::store((B*)a.dz + dense, k, dv);
                if (scaled) ds[v] += dv * EA::widen(cur.za[v]);
                EA::store((A*)a.dx + dense, k, dv * sc[v]);
            } else {
                const f32x8 zv = EA::widen(cur.za[v]), xv = EB::widen(cur.xb[v]), dy = EA::widen(cur.dy[v]);
                f32x8 dx, dz;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = zv[e], s = sigm(z), dsilu = s * (1.f + z * (1.f - s));
                    if (KIND == 1) {
                        dx[e] = dv[e] * (z * s);
                        dz[e] = dv[e] * xv[e] * dsilu;
                    } else {
                        dx[e] = dv[e];
                        dz[e] = dy[e] * w[v][e] * m[v][e] * dsilu;
                    }
                }
                EB::store((B*)a.dx + row * a.dx_stride + g0, k, dx);
                EA::store((A*)a.dz + row * a.dz_stride + g0, k, dz);
            }
        }
    }
    // this workgroup's sums over its rows
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && !scaled) break;
        f32x8(&s)[V] = k ? ds : dw;
        float* to = a.part + ((int64_t)k * a.nparts + blockIdx.x) * a.D + g0;
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
            if (wave || lane >= LANES) continue;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int o = 0; o < 3; ++o) {
                    const f32x4 lo = sums[((o * V + v) * 2) * 64 + lane], hi = sums[((o * V + v) * 2 + 1) * 64 + lane];
                    s[v] += __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) EW::store_cached(to, p.template cols<SPLIT>(v, n), s[v]);
    }
}

// dweight (blockIdx.y 0) and dscale (1) from the workgroups' partial sums.
__global__ __launch_bounds__(kSumThreads) void norm_sums_kernel(NormArgs a, int64_t n) {
    const int col = blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const float* part = a.part + (int64_t)blockIdx.y * a.nparts * a.D;
    const float s = column_sum(n, [&](int64_t t) { return col < a.D ? part[t * a.D + col] : 0.f; });
    if (threadIdx.x < kSumCols && col < a.D) (blockIdx.y ? a.dscale : a.dweight)[col] = s;
}

// Threads of a workgroup for rows of n columns with LANES lanes a team.
inline int norm_threads(int n, int V) { return (n + 64 * kVec * V - 1) / (64 * kVec * V) * 64; }

template <typename A, typename B, int KIND, int LANES, bool WIDE, int V>
hipError_t run_norm(const NormArgs& a, bool backward, hipStream_t stream) {
    const int threads = WIDE ? norm_threads(a.D / a.G, V) : 256;
    if (backward) {
        if (a.rows > 0) {
            hipLaunchKernelGGL((norm_backward_kernel<A, B, KIND, LANES, WIDE, V>), dim3(a.nparts, a.G), dim3(threads), 0,
                               stream, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL(norm_sums_kernel, dim3((a.D + kSumCols - 1) / kSumCols, a.dscale ? 2 : 1), dim3(kSumThreads), 0,
                           stream, a, (int64_t)(a.rows > 0 ? a.nparts : 0));
        return hipGetLastError();
    }
    const int64_t segs = a.rows * a.G, per = WIDE ? 1 : 256 / LANES;
    if (segs == 0) return hipSuccess;
    const int64_t blocks = std::min<int64_t>((segs + per - 1) / per, kMaxBlocks);
    hipLaunchKernelGGL((norm_forward_kernel<A, B, KIND, LANES, WIDE, V>), dim3((unsigned)blocks), dim3(threads), 0, stream,
                       a);
    return hipGetLastError();
}

// Vectors of 8 columns a lane: as few as up to 8 waves a row allow.
inline int norm_vectors(int n) { return n <= 4096 ? 1 : n <= 8192 ? 2 : 4; }

template <typename A, typename B, int KIND>
hipError_t by_columns(const NormArgs& a, bool backward, hipStream_t stream) {
    const int n = a.D / a.G;
    if (n <= 8 * kVec) return run_norm<A, B, KIND, 8, false, 1>(a, backward, stream);
    if (n <= 16 * kVec) return run_norm<A, B, KIND, 16, false, 1>(a, backward, stream);
    if (n <= 32 * kVec) return run_norm<A, B, KIND, 32, false, 1>(a, backward, stream);
    if (n <= 64 * kVec) return run_norm<A, B, KIND, 64, false, 1>(a, backward, stream);
    switch (norm_vectors(n)) {
        case 1: return run_norm<A, B, KIND, 64, true, 1>(a, backward, stream);
        case 2: return run_norm<A, B, KIND, 64, true, 2>(a, backward, stream);
        default: return run_norm<A, B, KIND, 64, true, 4>(a, backward, stream);
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

// Workgroups along the rows of the backward pass: what 256 compute units hold
// at once over all groups (16 waves each, 8 with more than one vector a lane),
// so that they run in one round; no more than there are rows for.
int32_t norm_parts(int64_t rows, int32_t D, int32_t G) {
    const int n = D / G, V = norm_vectors(n);
    int per = 1, waves = norm_threads(n, V) / 64;  // rows at once and waves of a workgroup
    if (n <= 64 * kVec) {
        per = 256 / (n <= 8 * kVec ? 8 : n <= 16 * kVec ? 16 : n <= 32 * kVec ? 32 : 64);
        waves = 4;
    }
    const int held = 256 * ((V == 1 ? 16 : 8) / waves);
    return (int32_t)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, std::max(1, held / G)));
}

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t stream) { return by_types<0>(a, false, stream); }
hipError_t launch_residual_norm_backward(const NormArgs& a, hipStream_t stream) { return by_types<0>(a, true, stream); }
hipError_t launch_gated_norm(const NormArgs& a, hipStream_t stream) {
    return a.norm_first ? by_types<2>(a, false, stream) : by_types<1>(a, false, stream);
}
hipError_t launch_gated_norm_backward(const NormArgs& a, hipStream_t stream) {
    return a.norm_first ? by_types<2>(a, true, stream) : by_types<1>(a, true, stream);
}

}  // namespace ssd
