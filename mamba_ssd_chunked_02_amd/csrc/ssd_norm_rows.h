// Shared by the norms: a row over a team of lanes, 8 columns a lane at a time, in
// either type.
#pragma once

#include <algorithm>

#include "ssd_column_sum.h"
#include "ssd_device.h"

namespace ssd {

constexpr int kVec = 8;
constexpr int kMaxWaves = 8;

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

__device__ inline float sum8(f32x8 v) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
// v - mean in the columns that are there, 0 in the others.
__device__ inline f32x8 away_from(f32x8 v, float mean, const Cols& k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = k.on[e >> 2] ? v[e] - mean : 0.f;
    return v;
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
    // Two sums; lds holds a pair for each wave of the workgroup.
    __device__ void sum2(float& u, float& v, float (*lds)[2]) const {
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) {
            u += __shfl_xor(u, d);
            v += __shfl_xor(v, d);
        }
        if constexpr (WIDE) {
            __syncthreads();
            if ((threadIdx.x & 63) == 0) {
                lds[threadIdx.x >> 6][0] = u;
                lds[threadIdx.x >> 6][1] = v;
            }
            __syncthreads();
            u = v = 0.f;
            for (int w = 0; w < (int)blockDim.x / 64; ++w) {
                u += lds[w][0];
                v += lds[w][1];
            }
        }
    }
};

// Threads of a workgroup for rows of n columns with LANES lanes a team.
inline int norm_threads(int n, int V) { return (n + 64 * kVec * V - 1) / (64 * kVec * V) * 64; }

// Vectors of 8 columns a lane: as few as up to 8 waves a row allow.
inline int norm_vectors(int n) { return n <= 4096 ? 1 : n <= 8192 ? 2 : 4; }

}  // namespace ssd
