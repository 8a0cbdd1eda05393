// Gradients of the causal depthwise conv1d (+ SiLU) on gfx950.  With
// v[t] = bias + sum_k w[k] xp[t + k] over the padded sequence
// xp = [conv state (K-1 rows); x] and out = silu(v):
//   dv[t]  = dy[t] silu'(v[t])                      (v recomputed from x)
//   dx[t]  = sum_k w[k] dv[t + K-1-k]               (inside the sequence)
//   dw[k]  = sum_t dv[t] xp[t + k],   db = sum_t dv[t]
// and what the final conv state's gradient adds to the last K-1 inputs.
// About 6K + 12 operations per element: an HBM stream (x and dy in, dx out).
// 65536 rows of 5376 channels, bf16, width 4, SiLU: 426 us, 5.0 TB/s.
//
// A lane owns 4 consecutive channels and walks a block of rows, sequence by
// sequence, in batches of kBatch.  The K-1 inputs and the K-1 dv that a batch
// shares with the next one stay in registers, and the next batch is in flight
// while one is computed, so a wave loads each of its rows once; the K-1 rows in
// front of them, the K-1 behind, whose dv its last dx need, and a last batch in
// flight are another wave's too (1.47 GB fetched for 1.41 at the shape above, in
// walks of 128 rows).  A batch inside its sequence and its walk takes a path with
// no test per row.
#include <algorithm>
#include <type_traits>

#include "ssd_column_sum.h"
#include "ssd_gated.h"

namespace ssd {

namespace {

constexpr int kBwdThreads = 256;
constexpr int kBatch = 4;
constexpr int kCh = 4;
constexpr int kWaveCh = 64 * kCh;

template <typename Y>
struct Part {
    const Y* p;
    int64_t stride;
};

// The gradient of the lane's 4 channels in row 0, and its row stride.
template <typename Y>
__device__ inline Part<Y> dy_part(const ConvBwdArgs& a, int c0) {
    int off = 0;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (p + 1 < a.nparts && c0 >= off + a.part_ch[p]) off += a.part_ch[p];
        else return {(const Y*)a.dy[p] + (c0 - off), a.part_ch[p]};
    }
    return {(const Y*)a.dy[2] + (c0 - off), a.part_ch[2]};
}

template <int K>
struct Taps4 {
    f32x4 w[K], b;
};

template <int K>
__device__ inline Taps4<K> load_taps4(const ConvBwdArgs& a, int c0) {
    Taps4<K> t;
#pragma unroll
    for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int k = 0; k < K; ++k) t.w[k][c] = a.weight[(int64_t)(c0 + c) * K + k];
    t.b = a.bias ? *(const f32x4*)(a.bias + c0) : f32x4{};
    return t;
}

// dv of one row from its K inputs and dy.
template <int K, bool SILU>
__device__ inline f32x4 dv_row(const Taps4<K>& t, const f32x4* h, f32x4 dy) {
    if constexpr (!SILU) return dy;
    f32x4 v = t.b;
#pragma unroll
    for (int k = 0; k < K; ++k) v += t.w[k] * h[k];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        const float s = sigmoid_f(v[c]);
        dy[c] *= s * (1.f + v[c] * (1.f - s));
    }
    return dy;
}

// The input j rows into the padded sequence [lo - (K-1), hi).
template <typename T, int K>
__device__ inline f32x4 padded_input(const ConvBwdArgs& a, int64_t s, RowRange q, int64_t j, int c0) {
    if (j < K - 1) return a.state_in ? Tr<T>::ld4((const T*)a.state_in + (s * (K - 1) + j) * a.C + c0) : f32x4{};
    return Tr<T>::ld4((const T*)a.x + (q.lo + j - (K - 1)) * a.C + c0);
}

// Gradient of the incoming state of sequence s: row j of it is an input of the
// tokens t < j + 1,
//   dstate[j] = sum over k <= j, j - k < length of w[k] dv[j - k],
// plus the final state's own gradient where the sequence is too short to
// have pushed the row out.
template <typename T, typename Y, int K, bool SILU>
__device__ inline void state_gradient(const ConvBwdArgs& a, int64_t s, int c0) {
    const RowRange q = seq_range(a.cu, a.L, a.T, s);
    const int64_t len = q.hi - q.lo;
    const Taps4<K> tp = load_taps4<K>(a, c0);
    const Part<Y> dyp = dy_part<Y>(a, c0);
    f32x4 ds[K - 1] = {};
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
        if (t >= len) break;
        f32x4 h[K];
#pragma unroll
        for (int k = 0; k < K; ++k) h[k] = padded_input<T, K>(a, s, q, t + k, c0);
        const f32x4 dv = dv_row<K, SILU>(tp, h, Tr<Y>::ld4(dyp.p + (q.lo + t) * dyp.stride));
#pragma unroll
        for (int k = 0; k + t < K - 1; ++k) ds[t + k] += tp.w[k] * dv;
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        // row j of the padded sequence is row j - len of the final state
        if (a.dstate_out && j >= len)
            ds[j] += Tr<T>::ld4((const T*)a.dstate_out + (s * (K - 1) + j - len) * a.C + c0);
        Tr<T>::st4((T*)a.dstate_in + (s * (K - 1) + j) * a.C + c0, ds[j]);
    }
}

// Workgroup bx < a.nblocks: a block of rows; the others: the incoming states'
// gradients, a sequence a wave.  Workgroups go to the 8 XCDs in turn: those of one
// XCD take the channel blocks of the same rows one after the other, so that it
// reads and writes whole rows (428 us at the shape below, 437 us with the row
// blocks in launch order).
template <typename T, typename Y, int K, bool SILU>
__global__ __launch_bounds__(kBwdThreads) void conv_backward_kernel(ConvBwdArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int ncb = (a.C + kWaveCh - 1) / kWaveCh;
    const int64_t bx = (int64_t)(blockIdx.x / 8 / ncb) * 8 + blockIdx.x % 8;
    const int c = (int)(blockIdx.x / 8 % ncb) * kWaveCh + lane * kCh;
    const bool on = c < a.C;
    const int c0 = on ? c : a.C - kCh;
    if (bx >= a.nblocks) {
        const int64_t stride = ((int64_t)gridDim.x / ncb - a.nblocks) * 4;
        for (int64_t s = (bx - a.nblocks) * 4 + wave; a.dstate_in && on && s < a.nseq; s += stride)
            state_gradient<T, Y, K, SILU>(a, s, c0);
        return;
    }
    const int rows = a.block_rows / 4;  // rows of a wave
    const int64_t r0 = min(bx * a.block_rows + wave * rows, a.T), r1 = min(r0 + rows, a.T);
    const RowRange live = live_rows(a.cu, a.nseq, a.T);
    const Taps4<K> tp = load_taps4<K>(a, c0);
    const Part<Y> dyp = dy_part<Y>(a, c0);
    const T* xb = (const T*)a.x + c0;
    T* dxb = (T*)a.dx + c0;
    f32x4 dw[K] = {}, db = {};
    typedef typename Raw<T>::type rawx;
    typedef typename Raw<Y>::type rawy;

    int64_t r = max(r0, live.lo);
    const int64_t end = min(r1, live.hi);
    while (r < end) {
        const int64_t s = seq_of(a.cu, a.nseq, a.L, r);
        const RowRange q = seq_range(a.cu, a.L, a.T, s);
        if (r < q.lo || r >= q.hi) {  // an invalid offset list
            ++r;
            continue;
        }
        const int64_t e = min(end, q.hi);  // this block's rows of the sequence: [r, e)
        rawx xn[kBatch];
        rawy yn[kBatch];
        // rows t + K-1 .. of the batch at t; behind the last row the last one again, unused
        auto load = [&](int64_t t) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t n = min(t + K - 1 + j, a.T - 1);
                xn[j] = __builtin_nontemporal_load((const rawx*)(xb + n * a.C));
                yn[j] = __builtin_nontemporal_load((const rawy*)(dyp.p + n * dyp.stride));
            }
        };
        load(r);
        // the inputs and dv of the rows r .. r + K-2
        f32x4 xh[K - 1], dvh[K - 1];
        {
            f32x4 in[2 * (K - 1)];
#pragma unroll
            for (int j = 0; j < 2 * (K - 1); ++j)
                in[j] = r + j - (K - 1) < q.hi ? padded_input<T, K>(a, s, q, r - q.lo + j, c0) : f32x4{};
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                xh[j] = in[K - 1 + j];
                dvh[j] = f32x4{};
                if (r + j >= q.hi) continue;
                dvh[j] = dv_row<K, SILU>(tp, in + j, Tr<Y>::ld4(dyp.p + (r + j) * dyp.stride));
                if (r + j >= e) continue;
                db += dvh[j];
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] += dvh[j] * in[j + k];
            }
        }
        // EDGE: the batch reaches the end of the block or of the sequence
        auto batch = [&](int64_t t, auto edge) {
            constexpr bool EDGE = decltype(edge)::value;
            f32x4 h[K - 1 + kBatch], d[K - 1 + kBatch];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                h[j] = xh[j];
                d[j] = dvh[j];
            }
            rawy y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                h[K - 1 + j] = Raw<T>::widen(xn[j]);
                y[j] = yn[j];
            }
            if (!EDGE) load(t + kBatch);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t n = t + K - 1 + j;
                d[K - 1 + j] = f32x4{};
                if (!EDGE || n < q.hi) {
                    const f32x4 v = dv_row<K, SILU>(tp, h + j, Raw<Y>::widen(y[j]));
                    d[K - 1 + j] = v;
                    if (!EDGE || n < e) {
                        db += v;
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k] += v * h[j + k];
                    }
                }
                if (EDGE && t + j >= e) continue;
                f32x4 dx = {};
#pragma unroll
                for (int k = 0; k < K; ++k) dx += tp.w[k] * d[j + K - 1 - k];
                // the final state holds the last K-1 inputs
                if (EDGE && a.dstate_out && t + j >= q.hi - (K - 1))
                    dx += Tr<T>::ld4((const T*)a.dstate_out + (s * (K - 1) + t + j - (q.hi - (K - 1))) * a.C + c0);
                if (on) __builtin_nontemporal_store(Tr<T>::narrow4(dx), (typename Tr<T>::v4*)(dxb + (t + j) * a.C));
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                xh[j] = h[kBatch + j];
                dvh[j] = d[kBatch + j];
            }
            if (EDGE) load(t + kBatch);
        };
        for (; r + kBatch + K - 1 <= e; r += kBatch) batch(r, std::false_type{});
        for (; r < e; r += kBatch) batch(r, std::true_type{});
        r = e;
    }
    // the workgroup's sums: waves 1..3 through LDS, added in order
    __shared__ f32x4 sums[3][K + 1][64];
    if (wave) {
#pragma unroll
        for (int k = 0; k < K; ++k) sums[wave - 1][k][lane] = dw[k];
        sums[wave - 1][K][lane] = db;
    }
    __syncthreads();
    if (wave || !on) return;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        f32x4 v = k < K ? dw[k < K ? k : 0] : db;
#pragma unroll
        for (int o = 0; o < 3; ++o) v += sums[o][k][lane];
        *(f32x4*)(a.part + (bx * (K + 1) + k) * a.C + c0) = v;
    }
}

// dweight [C, K] and dbias [C] from the workgroups' sums.
template <int K>
__global__ __launch_bounds__(kSumThreads) void conv_backward_sum_kernel(ConvBwdArgs a, int64_t n) {
    const int c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, k = blockIdx.y;
    const float s = column_sum(n, [&](int64_t t) { return c < a.C ? a.part[(t * (K + 1) + k) * a.C + c] : 0.f; });
    if (threadIdx.x >= kSumCols || c >= a.C) return;
    if (k < K) a.dweight[(int64_t)c * K + k] = s;
    else if (a.dbias) a.dbias[c] = s;
}

template <typename T, typename Y, int K, bool SILU>
hipError_t run_conv_backward(ConvBwdArgs a, hipStream_t stream) {
    const int64_t ncb = (a.C + kWaveCh - 1) / kWaveCh;
    const int64_t states = a.dstate_in ? std::min<int64_t>((a.nseq + 3) / 4, std::max<int64_t>(1, (1 << 22) / ncb)) : 0;
    a.nblocks = a.T > 0 ? a.nblocks : 0;
    if (a.nblocks + states > 0) {
        hipLaunchKernelGGL((conv_backward_kernel<T, Y, K, SILU>),
                           dim3((unsigned)((a.nblocks + states + 7) / 8 * 8 * ncb)),
                           dim3(kBwdThreads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((conv_backward_sum_kernel<K>), dim3((unsigned)((a.C + kSumCols - 1) / kSumCols), K + 1),
                       dim3(kSumThreads), 0, stream, a, (int64_t)a.nblocks);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t by_width(const ConvBwdArgs& a, hipStream_t stream) {
    switch (a.K) {
        case 2: return a.silu ? run_conv_backward<T, Y, 2, true>(a, stream) : run_conv_backward<T, Y, 2, false>(a, stream);
        case 3: return a.silu ? run_conv_backward<T, Y, 3, true>(a, stream) : run_conv_backward<T, Y, 3, false>(a, stream);
        case 4: return a.silu ? run_conv_backward<T, Y, 4, true>(a, stream) : run_conv_backward<T, Y, 4, false>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

// Rows of a workgroup: 512 for long batches, fewer (in steps of 32, two batches
// a wave) where that leaves the chip short of 1024 workgroups.
void conv_backward_blocks(int64_t T, int32_t C, int32_t* nblocks, int32_t* block_rows) {
    const int64_t cb = (C + kWaveCh - 1) / kWaveCh;
    int64_t rows = T * cb / 1024 / 32 * 32;
    rows = std::max<int64_t>(32, std::min<int64_t>(512, rows));
    *block_rows = (int32_t)rows;
    *nblocks = (int32_t)std::max<int64_t>(1, (T + rows - 1) / rows);
}

hipError_t launch_conv1d_backward(const ConvBwdArgs& a, hipStream_t stream) {
    if (a.dtype == 1) return a.y_f32 ? by_width<bf16_t, float>(a, stream) : by_width<bf16_t, bf16_t>(a, stream);
    return a.y_f32 ? by_width<float, float>(a, stream) : by_width<float, bf16_t>(a, stream);
}

}  // namespace ssd
