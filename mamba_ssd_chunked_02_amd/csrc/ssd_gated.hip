// Gated linear recurrence on gfx950: per sequence and channel, with gates
// computed from two logits of every token,
//   log a_t = -rate softplus(lam) sigmoid(r_t)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t,
// and its gradients.  About 40 fp32 operations (6 of them quarter rate) and 8
// bytes (bf16) an element: an HBM stream, with the vector ALU close behind
// (busy 80% of the time forward).  Measured: 49152 rows of 8192 channels forward
// 627 us, 5.1 TB/s; 65536 rows of 2560 channels forward and backward 842 us, 4.4
// TB/s.
//
// The token axis of the whole batch is cut into tiles of 128 rows (64 backward)
// whatever the sequences' lengths; a sequence start inside a tile resets the
// state there.  A step is the map h -> a h + b, and a run of steps is again
// such a map (P, H): state at the end = P * (state before) + H.  A reset in a
// run makes P negative (its sign bit is the mark; P is never negative
// otherwise), so that nothing of the earlier sequence, NaN and infinities
// included, gets through a multiplication by 0.
//
// One pass over the data: a workgroup holds its tile in registers, publishes
// the tile's map, folds the maps of the tiles before it into the state that
// enters its own, and finishes.  Tiles go in groups of 8: a tile folds the maps
// of its group's earlier tiles, in order, onto the state entering the group,
// which the last tile of the group before publishes.  So the order of every sum
// is fixed, and only one step in 8 tiles is a chain.
//   Why the waits end: the tiles of a channel block are handed out in order by
// a counter, so every tile that a workgroup waits for belongs to a workgroup
// that runs already, and a tile's map is published before its workgroup waits
// for anything.  The state entering a group waits only for earlier tiles.
//
// A decay near 1 is rounded to fp32 (half of 2^-24), but the factor P of a run of
// rows comes from the sum of its log a and so has one such rounding, not one a
// row.  Those of the runs do add up where the gates are constant: at |log a| =
// 8.8e-8 a run of 8 rows a state is 2.3e-4 off after 65536 tokens, and below 2^-25
// a run nothing decays.  1 - a^2 comes from a - 1, which is computed by itself.
#include <algorithm>
#include <type_traits>

#include "ssd_column_sum.h"
#include "ssd_gated.h"

namespace ssd {

namespace {

constexpr int kLaneCh = 4;                      // channels per lane
constexpr int kSegLanes = 16;                   // lanes across the channels of a row
constexpr int kTileCh = kLaneCh * kSegLanes;    // channels per workgroup
constexpr int kFwdTile = 128, kBwdTile = kGatedStateRows;  // rows per tile
constexpr int kGroup = 8;                       // tiles per group of the carry
constexpr int kFwdRows = 8, kBwdRows = 4;       // rows per run (per lane)
constexpr uint64_t kNotYet = ~(uint64_t)0;      // a published word that is not there yet
static_assert(kFwdTile % kGatedStateRows == 0 && kGatedStateRows % kFwdRows == 0, "saved states fall on runs");

__device__ inline bool is_reset(float P) { return __builtin_bit_cast(int, P) < 0; }

// The run (P, H) applied to a state.
__device__ inline float advance(float P, float H, float h) { return is_reset(P) ? H : __builtin_fmaf(P, h, H); }
// The factor of a run followed by one with factor P.
__device__ inline float chain(float before, float P) { return is_reset(P) ? -1.f : before * P; }

__device__ inline float nan_to_positive(float P) {
    return P != P ? __builtin_bit_cast(float, 0x7fc00000) : P;
}

// A pair of floats as one word that is stored and loaded whole, past the
// caches of one XCD.  hi is no NaN with its sign bit set, so never kNotYet.
__device__ inline void publish(uint64_t* p, float hi, float lo) {
    const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, hi) << 32 | __builtin_bit_cast(uint32_t, lo);
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t look(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline bool there(uint64_t v) { return (uint32_t)(v >> 32) != 0xffffffffu; }
__device__ inline float hi_of(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)(v >> 32)); }
__device__ inline float lo_of(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)v); }

// Before the pass: the published words set to kNotYet and the counters to 0;
// for a packed batch the boundary bits, and the states of sequences without
// tokens (their state passes through: out = in).
__global__ __launch_bounds__(256) void gated_plan_kernel(GatedArgs a, GatedPlan pl) {
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    const int64_t me = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t k = me; k < pl.nwords; k += stride) pl.words[k] = kNotYet;
    for (int64_t k = me; k < pl.ncounters; k += stride) pl.counters[k] = 0;
    const int64_t nruns = (a.T + kBitRows - 1) / kBitRows;
    const RowRange live = live_rows(a.cu, a.nseq, a.T);
    for (int64_t k = me; pl.bits && k < nruns; k += stride)
        pl.bits[k] = packed_boundaries(a.cu, a.nseq, live, k * kBitRows);
    if (!pl.out) return;
    const int64_t waves = stride / 64, lane = me & 63;
    for (int64_t s = me / 64; s < a.nseq; s += waves) {
        const RowRange q = seq_range(a.cu, a.L, a.T, s);
        if (q.hi > q.lo) continue;
        for (int64_t c = lane; c < a.C; c += 64) pl.out[s * a.C + c] = pl.in ? pl.in[s * a.C + c] : 0.f;
    }
}

// What a lane has of its run of rows: the place, the boundary bits (of live rows)
// and the live rows (bit j).  plain: no run of the wave has a boundary or a row that is
// not live, and so none of the tests per row is needed.
template <int ROWS, int TILE>
struct Run {
    int64_t tile0;   // the tile's first row
    int row;         // the run's first row in the tile
    int c0;          // first channel (clamped into the row)
    bool on;         // the lane's channels exist
    int plain;       // (a scalar)
    uint32_t bits, live;
    __device__ int64_t t(int j) const { return tile0 + row + j; }
    __device__ bool start(int j) const { return bits >> j & 1; }
    __device__ bool end(int j) const { return bits >> (16 + j) & 1; }
    __device__ bool has(int j) const { return live >> j & 1; }
    __device__ bool any_start() const { return bits & 0xffff; }
    __device__ bool any_end() const { return bits >> 16; }

    __device__ Run(const GatedArgs& a, int64_t tile, int cb) {
        tile0 = tile * TILE;
        row = (int)(threadIdx.x / kSegLanes) * ROWS;
        const int c = cb * kTileCh + (threadIdx.x % kSegLanes) * kLaneCh;
        on = c < a.C;
        c0 = on ? c : a.C - kLaneCh;
        if (!a.cu) {
            // rows < 2^31; the whole tile between two boundaries, or not
            const uint32_t p = (uint32_t)tile0 % (uint32_t)a.L;
            if (p && a.L - p > TILE) {
                bits = 0;
                live = (1u << ROWS) - 1;
                plain = 1;
                return;
            }
        }
        const RunBits r = run_bits<ROWS>(a.cu, a.bits, a.nseq, a.L, a.T, t(0));
        bits = r.bits;
        live = r.live;
        plain = __builtin_amdgcn_readfirstlane(__all(bits == 0 && live == (1u << ROWS) - 1));
    }
};

// Row j of the run in a [rows, stride] tensor: a base that is the same for the
// whole workgroup plus a 32-bit offset of the lane that is the same for every
// j (strides are at most 2^22 elements).
template <typename T>
__device__ inline T* at_row(T* p, int64_t row0, int64_t stride, uint32_t bytes) {
    return (T*)((char*)(p + row0 * stride) + bytes);
}

// The data is read once and written once: streaming loads and stores.  A tile
// that reaches past the last row reads that row instead.
template <typename T, int ROWS, int TILE>
__device__ inline void load_rows(const GatedArgs& a, const Run<ROWS, TILE>& u, const void* p, int64_t stride,
                                 typename Raw<T>::type (&v)[ROWS]) {
    typedef typename Raw<T>::type raw;
    T* const q = (T*)const_cast<void*>(p);
    if (u.tile0 + TILE <= a.T) {
        const uint32_t bytes = ((uint32_t)u.row * (uint32_t)stride + (uint32_t)u.c0) * sizeof(T);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) v[j] = __builtin_nontemporal_load((const raw*)at_row(q, u.tile0 + j, stride, bytes));
    } else {
        const int last = (int)(a.T - 1 - u.tile0);
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
            v[j] = *(const raw*)at_row(
                q, u.tile0, stride, ((uint32_t)min(u.row + j, last) * (uint32_t)stride + (uint32_t)u.c0) * sizeof(T));
    }
}

template <typename T, int ROWS, int TILE>
__device__ inline void store_row(const Run<ROWS, TILE>& u, void* p, int64_t stride, int j, f32x4 v) {
    const uint32_t bytes = ((uint32_t)u.row * (uint32_t)stride + (uint32_t)u.c0) * sizeof(T);
    __builtin_nontemporal_store(Tr<T>::narrow4(v), (typename Tr<T>::v4*)at_row((T*)p, u.tile0 + j, stride, bytes));
}

__device__ inline int64_t state_at(const GatedArgs& a, int64_t row, int c0) {
    return seq_of(a.cu, a.nseq, a.L, row) * a.C + c0;
}

// Rows that are not live become steps that change nothing: log a = 0, x = 0.
template <typename T, int ROWS, int TILE>
__device__ inline void idle_rows(const Run<ROWS, TILE>& u, typename Raw<T>::type (&xv)[ROWS], typename Raw<T>::type (&rv)[ROWS],
                                 typename Raw<T>::type (&iv)[ROWS]) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
        if (!u.has(j)) {
            xv[j] = iv[j] = Raw<T>::all(0.f);
            rv[j] = Raw<T>::all(-__builtin_inff());
        }
}

__device__ inline f32x4 seq_state(const GatedArgs& a, const float* st, int64_t row, int c0) {
    return st ? *(const f32x4*)(st + state_at(a, row, c0)) : f32x4{};
}

// The value is computed here and kept, and what it was computed from is
// forgotten: without this the compiler keeps every row's intermediate values
// alive for a later use of the same expression, 40 to 90 registers more.
template <typename V>
__device__ inline void pin(V& v) {
#pragma unroll
    for (int c = 0; c < (int)(sizeof(V) / 4); ++c) {
        auto t = v[c];
        asm volatile("" : "+v"(t));
        v[c] = t;
    }
}

// One row: the gates, the held decay, a and b of four channels.
template <typename T>
struct Step {
    f32x4 sr, si, w, a, b;
    __device__ Step(f32x4 k, bool slow, typename Raw<T>::type xv, typename Raw<T>::type rv, typename Raw<T>::type iv) {
        const f32x4 x = Raw<T>::widen(xv), r = Raw<T>::widen(rv), i = Raw<T>::widen(iv);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sr[c] = sigmoid_f(r[c]);
            si[c] = sigmoid_f(i[c]);
        }
        Decay d;
        d.from_log(k * sr, slow);
        w = d.w;
        a = d.a;
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = __builtin_amdgcn_sqrtf(d.m[c]) * si[c] * x[c];
    }
};

// At a sequence's first row the initial state goes into b and the state before
// it counts as 0: H goes on from (a, b) of row j.
template <int ROWS, int TILE>
__device__ inline void take_row(const GatedArgs& a, const Run<ROWS, TILE>& u, int j, f32x4 av, f32x4& b, f32x4& H) {
    if (!u.plain)
        if (u.start(j)) {
            b += av * seq_state(a, a.init, u.t(j), u.c0);
            H = f32x4{};
        }
    H = av * H + b;
}

__device__ inline int slow_wave(f32x4 k) {
    return __builtin_amdgcn_readfirstlane(!__any(fminf(fminf(k[0], k[1]), fminf(k[2], k[3])) < kSlowDecay));
}

// A run's factor from its sum of log a.
__device__ inline f32x4 run_factor(f32x4 S, bool reset) {
    f32x4 P;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        P[c] = reset ? -1.f : nan_to_positive(__builtin_amdgcn_exp2f(S[c] * 1.44269504088896341f));
    return P;
}

// The workgroup's channel block.  Workgroups go to the 8 XCDs in turn; by_rows
// gives consecutive workgroups of one XCD consecutive channel blocks, so that
// an XCD reads and writes whole rows instead of every eighth 128 bytes of them
// (49152 rows of 8192 channels 631 us, channel blocks in launch order 691 us;
// forward and backward over 65536 rows of 2560 channels 842 against 920 us).  A
// pass of a single round of workgroups is quicker in launch order (4096 rows of
// 1536 channels 18.7 against 19.8 us).
__device__ inline int channel_block(const GatedPass& ps) {
    return (ps.by_rows ? blockIdx.x / 8 : blockIdx.x) % ps.nblocks;
}

// Which tile this workgroup has: the channel block's next one, in the pass's
// order (behind the last tile, where there are more workgroups than tiles: none).
__device__ inline int64_t next_tile(const GatedPass& ps, int cb, uint32_t* slot) {
    if (!ps.counters) return 0;
    if (threadIdx.x == 0) *slot = atomicAdd(ps.counters + cb * kGatedCounterStride, 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*slot);
}

// The runs' maps in LDS, folded in order (REV: from the last run back).
template <int RUNS, bool REV>
struct Fold {
    const float *P, *H;  // [RUNS][kTileCh]
    __device__ static int at(int s) { return (REV ? RUNS - 1 - s : s) * kTileCh; }
    // the tile's own map
    __device__ void map(int ch, float& Pt, float& Ht) const {
        Pt = 1.f;
        Ht = 0.f;
#pragma unroll 4
        for (int s = 0; s < RUNS; ++s) {
            const float p = P[at(s) + ch];
            Ht = advance(p, H[at(s) + ch], Ht);
            Pt = chain(Pt, p);
        }
    }
    // H replaced by the state entering each run
    __device__ void enter(int ch, float h) const {
        enter(ch, h, [](int, float) {});
    }
    // seen(s, h): run s is entered with h
    template <typename F>
    __device__ void enter(int ch, float h, F seen) const {
#pragma unroll 4
        for (int s = 0; s < RUNS; ++s) {
            seen(s, h);
            float* const to = const_cast<float*>(H) + at(s) + ch;
            const float n = advance(P[at(s) + ch], *to, h);
            *to = h;
            h = n;
        }
    }
};

// The tile's own map, for the later tiles of its group (by wave 0; the last
// tile's goes into the state entering the next group instead).
__device__ inline void publish_map(const GatedPass& ps, int64_t ord, int chan, int C, float Pt, float Ht) {
    if (chan < C && ord % kGroup < kGroup - 1 && ord + 1 < ps.ntiles) publish(ps.maps + ord * C + chan, Pt, Ht);
}

// The state entering tile `ord` (counted in the pass's order) for channel
// chan = channel block * 64 + lane, valid in wave 0.  (Pt, Ht): the tile's own
// map, in wave 0.  Every wave calls it; group_s: [kGroup][kTileCh] pairs.
template <int WAVES>
__device__ inline float enter_tile(const GatedPass& ps, int64_t ord, int chan, int C, float Pt, float Ht, f32x2* group_s) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool on = chan < C;
    const int at = on ? chan : 0;  // a lane without a channel reads there and waits for nothing
    const int p = (int)(ord % kGroup);
    const int64_t g = ord / kGroup;
    // wave 0 asks for the group's entry along with the maps
    uint64_t e = wave == 0 && g > 0 ? look(ps.entry + g * C + at) : 0;
    // the maps of the group's earlier tiles: wave w takes kGroup / WAVES of them
    constexpr int kEach = kGroup / WAVES;
    static_assert(kEach * WAVES == kGroup && WAVES >= 2, "every wave takes as many maps");
    const int j0 = wave * kEach;
    if (j0 < p) {
        const uint64_t* m = ps.maps + (g * kGroup + j0) * C + at;
        uint64_t v[kEach];
        while (true) {
            bool ready = true;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                v[j] = j0 + j < p ? look(m + (int64_t)j * C) : 0;
                ready &= !on || there(v[j]);
            }
            if (__all(ready)) break;
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) group_s[(j0 + j) * kTileCh + lane] = f32x2{hi_of(v[j]), lo_of(v[j])};
    }
    __syncthreads();
    if (wave) return 0.f;
    float Pp = 1.f, h = 0.f;
    for (int j = 0; j < p; ++j) {
        const f32x2 m = group_s[j * kTileCh + lane];
        h = advance(m[0], m[1], h);
        Pp = chain(Pp, m[0]);
    }
    // a sequence that starts in the group needs nothing from before it
    if (g > 0 && !__all(!on || is_reset(Pp))) {
        while (!__all(!on || there(e))) {
            __builtin_amdgcn_s_sleep(1);
            e = look(ps.entry + g * C + at);
        }
        h = advance(Pp, h, lo_of(e));
    }
    if (on && p == kGroup - 1 && ord + 1 < ps.ntiles) publish(ps.entry + (g + 1) * C + chan, 0.f, advance(Pt, Ht, h));
    return h;
}

// ------------------------------------------------------------------ forward
template <typename T, typename Y>
__global__ __launch_bounds__(kFwdTile / kFwdRows * kSegLanes) void gated_forward_kernel(GatedArgs a, GatedPass ps) {
    constexpr int R = kFwdRows, kRuns = kFwdTile / R;
    __shared__ uint32_t slot;
    __shared__ float k_s[kTileCh];
    __shared__ f32x4 P_s[kRuns][kSegLanes], H_s[kRuns][kSegLanes];
    __shared__ f32x2 group_s[kGroup * kTileCh];
    const int seg = threadIdx.x / kSegLanes, ln = threadIdx.x % kSegLanes;
    const int cb = channel_block(ps);
    if (threadIdx.x < kTileCh)
        k_s[threadIdx.x] = decay_factor(a.lam[min(cb * kTileCh + (int)threadIdx.x, a.C - 1)], a.rate);
    const int64_t tile = next_tile(ps, cb, &slot);
    if (tile >= ps.ntiles) return;  // the whole workgroup
    const Run<R, kFwdTile> u(a, tile, cb);
    typename Raw<T>::type xv[R], rv[R], iv[R];
    load_rows<T>(a, u, a.r, a.r_stride, rv);
    load_rows<T>(a, u, a.i, a.i_stride, iv);
    load_rows<T>(a, u, a.x, a.x_stride, xv);
    __syncthreads();
    const f32x4 k = *(const f32x4*)(k_s + ln * kLaneCh);

    if (!u.plain) idle_rows<T>(u, xv, rv, iv);
    const int slow = slow_wave(k);
    f32x4 av[R], b[R], S = {}, H = {};
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const Step<T> st(k, slow, xv[j], rv[j], iv[j]);
        S += st.sr;
        av[j] = st.a;
        b[j] = st.b;
        take_row(a, u, j, av[j], b[j], H);
        pin(av[j]);
        pin(b[j]);
        pin(S);
    }
    S *= k;
    P_s[seg][ln] = run_factor(S, u.any_start());
    H_s[seg][ln] = H;
    __syncthreads();
    const Fold<kRuns, false> fold{(const float*)P_s, (const float*)H_s};
    const int ch = threadIdx.x & 63, chan = cb * kTileCh + ch;
    float Pt = 1.f, Ht = 0.f, h0 = 0.f;
    if (ps.counters) {
        if (threadIdx.x < kTileCh) {
            fold.map(ch, Pt, Ht);
            publish_map(ps, tile, chan, a.C, Pt, Ht);
        }
        h0 = enter_tile<kRuns / 4>(ps, tile, chan, a.C, Pt, Ht, group_s);
    }
    if (threadIdx.x < kTileCh) {
        constexpr int kEvery = kGatedStateRows / R, kHere = kFwdTile / kGatedStateRows;
        if (a.states_out && chan < a.C)
            fold.enter(ch, h0, [&](int s, float h) {
                const int64_t at = tile * kHere + s / kEvery;
                if (s % kEvery == 0 && at * kGatedStateRows < a.T) a.states_out[at * a.C + chan] = h;
            });
        else fold.enter(ch, h0);
    }
    __syncthreads();
    if (!u.on) return;
    f32x4 h = H_s[seg][ln];
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (u.plain) {
            h = av[j] * h + b[j];
            store_row<Y>(u, a.y, a.C, j, h);
        } else if (u.has(j)) {
            h = av[j] * (u.start(j) ? f32x4{} : h) + b[j];
            store_row<Y>(u, a.y, a.C, j, h);
            if (a.final_state && u.end(j)) *(f32x4*)(a.final_state + state_at(a, u.t(j), u.c0)) = h;
        }
    }
}

// ------------------------------------------------------------------ backward
// With q_{t+1} = a_{t+1} g_{t+1} the adjoint reaching token t from behind
// (dfinal at a sequence's last token): g_t = dy_t + q_{t+1}, and
//   dx = g beta sig(i),  di = g beta sig(i) (1 - sig(i)) x,
//   d log a = g (a h_{t-1} - a^2 / beta sig(i) x),
//   dr = dloga loga (1 - sig(r)),  dlam = sum dloga loga sigmoid(lam)/softplus(lam),
//   dinit = q at a sequence's first token.
// h_{t-1} is recomputed in fp32 from the state entering the tile, which the
// forward pass kept; the adjoint is carried over the tiles in reverse order.
// 4 rows a lane and 64-row tiles, so that 4 workgroups a compute unit wait apart
// (8 rows a lane at half the waves 904 against 840 us).  At the 128 registers of
// four waves the bf16 kernel spills 3 of them (7 with fp32 dy; 16 and 32 bytes of
// scratch a lane): 1.16 GB written for 1.04 at 65536 rows of 2560 channels, and
// still quicker than three waves without (906 us).  fp32 rows take more (146) and are
// quicker with 3 (103 against 114 us, 8083 rows of 776 channels).
template <typename T, typename Y>
__global__ __launch_bounds__(kBwdTile / kBwdRows * kSegLanes, sizeof(T) == 2 ? 4 : 3)
void gated_backward_kernel(GatedArgs a, GatedPass ps, float* dlam_part) {
    constexpr int R = kBwdRows, kRuns = kBwdTile / R;
    __shared__ uint32_t slot;
    __shared__ float k_s[kTileCh];
    __shared__ f32x4 P_s[kRuns][kSegLanes], H_s[kRuns][kSegLanes], R_s[kRuns][kSegLanes], Q_s[kRuns][kSegLanes];
    __shared__ f32x2 group_s[kGroup * kTileCh];
    const int seg = threadIdx.x / kSegLanes, ln = threadIdx.x % kSegLanes;
    const int cb = channel_block(ps);
    if (threadIdx.x < kTileCh)
        k_s[threadIdx.x] = decay_factor(a.lam[min(cb * kTileCh + (int)threadIdx.x, a.C - 1)], a.rate);
    const int64_t ord = next_tile(ps, cb, &slot), tile = ps.ntiles - 1 - ord;
    if (tile < 0) return;  // the whole workgroup
    const Run<R, kBwdTile> u(a, tile, cb);
    typename Raw<T>::type xv[R], rv[R], iv[R];
    typename Raw<Y>::type dv[R];
    load_rows<T>(a, u, a.r, a.r_stride, rv);
    load_rows<Y>(a, u, a.dy, a.C, dv);
    load_rows<T>(a, u, a.i, a.i_stride, iv);
    load_rows<T>(a, u, a.x, a.x_stride, xv);
    const int ch = threadIdx.x & 63, chan = cb * kTileCh + ch;
    // wave 1 folds the states, wave 0 the adjoints
    const float state0 = threadIdx.x >> 6 == 1 && chan < a.C ? a.states_in[tile * a.C + chan] : 0.f;
    __syncthreads();
    const f32x4 k = *(const f32x4*)(k_s + ln * kLaneCh);
    const int slow = slow_wave(k);
    if (!u.plain) idle_rows<T>(u, xv, rv, iv);
    // first what the adjoint's map needs: the decays and dy
    f32x4 w[R], b[R], sr[R], si[R], S = {}, H = {}, Q = {};
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const f32x4 r = Raw<T>::widen(rv[j]);
#pragma unroll
        for (int c = 0; c < 4; ++c) sr[j][c] = sigmoid_f(r[c]);
        S += sr[j];
        Decay d;
        d.from_log(k * sr[j], slow);
        w[j] = d.w;
        pin(sr[j]);
        pin(w[j]);
        pin(S);
    }
    S *= k;
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
        f32x4 g = Raw<Y>::widen(dv[j]);
        if (!u.plain) {
            if (!u.has(j)) continue;
            if (u.end(j)) Q = seq_state(a, a.dfinal, u.t(j), u.c0);
        }
        Q = decay_of(w[j], slow) * (Q + g);
        pin(w[j]);
        pin(dv[j]);
    }
    R_s[seg][ln] = run_factor(S, u.any_end());
    Q_s[seg][ln] = Q;
    __syncthreads();
    const Fold<kRuns, false> states{(const float*)P_s, (const float*)H_s};
    const Fold<kRuns, true> adjoints{(const float*)R_s, (const float*)Q_s};
    float Rt = 1.f, Qt = 0.f, q0 = 0.f;
    if (ps.counters && threadIdx.x < kTileCh) {
        adjoints.map(ch, Rt, Qt);
        publish_map(ps, ord, chan, a.C, Rt, Qt);
    }
    // then the states, while the earlier tiles' maps arrive
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const f32x4 x = Raw<T>::widen(xv[j]), i = Raw<T>::widen(iv[j]);
        Decay d;
        d.from_held(w[j], slow);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            si[j][c] = sigmoid_f(i[c]);
            b[j][c] = __builtin_amdgcn_sqrtf(d.m[c]) * si[j][c] * x[c];
        }
        take_row(a, u, j, d.a, b[j], H);
        pin(si[j]);
        pin(b[j]);
        pin(w[j]);
        pin(xv[j]);
    }
    P_s[seg][ln] = run_factor(S, u.any_start());
    H_s[seg][ln] = H;
    __syncthreads();
    if (threadIdx.x >> 6 == 1) states.enter(ch, state0);
    if (ps.counters) q0 = enter_tile<kRuns / 4>(ps, ord, chan, a.C, Rt, Qt, group_s);
    if (threadIdx.x < kTileCh) adjoints.enter(ch, q0);
    __syncthreads();

    f32x4 h = H_s[seg][ln], q = Q_s[seg][ln], dl = {};
    // b: the state before each row from here on
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (!u.plain && u.start(j)) h = f32x4{};
        const f32x4 n = decay_of(w[j], slow) * h + b[j];
        b[j] = h;
        if (!u.plain && u.start(j)) b[j] = seq_state(a, a.init, u.t(j), u.c0);
        h = n;
        pin(w[j]);
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
        if (!u.plain) {
            if (!u.has(j)) continue;
            if (u.end(j)) q = seq_state(a, a.dfinal, u.t(j), u.c0);
        }
        const f32x4 x = Raw<T>::widen(xv[j]);
        const f32x4 g = q + Raw<Y>::widen(dv[j]);
        Decay d;
        d.from_held(w[j], slow);
        q = d.a * g;
        f32x4 dx, di, dr;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // 1 - a^2 = 0 only where log a is 0, and its square root's reciprocal meets that factor below;
            // a floor (the least normal number) keeps their product 0 (a NaN passes)
            const float m = d.m[c] < 0x1p-126f ? 0x1p-126f : d.m[c];
            const float u = __builtin_amdgcn_rsqf(m) * si[j][c];  // sig(i) / beta
            const float dl0 = q[c] * __builtin_fmaf(-d.a[c] * u, x[c], b[j][c]) * sr[j][c];  // dloga loga / k
            dx[c] = g[c] * (d.m[c] * u);
            di[c] = dx[c] * __builtin_fmaf(-x[c], si[j][c], x[c]);
            dr[c] = dl0 * __builtin_fmaf(-k[c], sr[j][c], k[c]);
            dl[c] += dl0;
        }
        pin(q);
        pin(dl);
        if (u.on) {
            store_row<T>(u, a.dx, a.dx_stride, j, dx);
            store_row<T>(u, a.dr, a.dr_stride, j, dr);
            store_row<T>(u, a.di, a.di_stride, j, di);
            if (!u.plain && a.dinit && u.start(j)) *(f32x4*)(a.dinit + state_at(a, u.t(j), u.c0)) = q;
        }
    }
    __syncthreads();
    P_s[seg][ln] = dl * k;
    __syncthreads();
    if (threadIdx.x < kTileCh) {
        float s = 0.f;
#pragma unroll 8
        for (int j = 0; j < kRuns; ++j) s += ((const float*)P_s)[j * kTileCh + ch];
        if (chan < a.C) dlam_part[tile * a.C + chan] = s;
    }
}

// dlam from the tiles' sums.
__global__ __launch_bounds__(kSumThreads) void gated_dlam_kernel(GatedArgs a, int64_t ntiles, const float* part,
                                                                 float* dlam) {
    const int ch = blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const float s = column_sum(ntiles, [&](int64_t t) { return ch < a.C ? part[t * a.C + ch] : 0.f; });
    if (threadIdx.x >= kSumCols || ch >= a.C) return;
    // sigmoid(lam) / softplus(lam): 1 towards minus infinity, where both vanish
    const float lam = a.lam[ch], sp = softplus_f(lam);
    dlam[ch] = s * (sp < 1e-30f ? 1.f : (1.f / (1.f + expf(-lam))) / sp);
}

// ------------------------------------------------------------------ one token
template <typename T, typename Y>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedArgs a, const float* state, float* state_out) {
    const int64_t quads = a.C / kLaneCh;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < a.nseq * quads; id += (int64_t)gridDim.x * 256) {
        const int64_t n = id / quads;
        const int c0 = (int)(id - n * quads) * kLaneCh;
        f32x4 h = *(const f32x4*)(state + n * a.C + c0), k = *(const f32x4*)(a.lam + c0);
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = decay_factor(k[c], a.rate);
        typedef typename Raw<T>::type raw;
        const Step<T> st(k, false, *(const raw*)((const T*)a.x + n * a.x_stride + c0),
                         *(const raw*)((const T*)a.r + n * a.r_stride + c0),
                         *(const raw*)((const T*)a.i + n * a.i_stride + c0));
        h = st.a * h + st.b;
        *(f32x4*)(state_out + n * a.C + c0) = h;
        Tr<Y>::st4((Y*)a.y + n * a.C + c0, h);
    }
}

inline int64_t blocks_of(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Workgroups of a pass; by rows, the XCDs take equal numbers of tiles.
inline int64_t pass_blocks(const GatedPass& ps) {
    return (ps.by_rows ? (ps.ntiles + 7) / 8 * 8 : ps.ntiles) * ps.nblocks;
}

// Clears what the pass publishes and plans a packed batch; nothing to do for
// a dense batch of one tile.
hipError_t run_plan(GatedArgs& a, const GatedLayout& lay, char* ws, const float* in, float* out, GatedPass* ps,
                    hipStream_t stream) {
    const bool many = lay.ntiles > 1;
    *ps = GatedPass{lay.ntiles, (int32_t)blocks_of(a.C, kTileCh), 0, nullptr, nullptr, nullptr};
    ps->by_rows = many && lay.ntiles * ps->nblocks > 1024;  // more than a round of 4 workgroups a compute unit
    GatedPlan pl{nullptr, 0, nullptr, 0, nullptr, in, nullptr};
    if (many) {
        pl.words = ps->maps = (uint64_t*)(ws + lay.maps);
        ps->entry = ps->maps + lay.ntiles * a.C;
        pl.nwords = (lay.ntiles + lay.ngroups) * a.C;
        pl.counters = ps->counters = (uint32_t*)(ws + lay.counters);
        pl.ncounters = (int64_t)ps->nblocks * kGatedCounterStride;
    }
    if (a.cu && a.T > 0) a.bits = pl.bits = (uint32_t*)(ws + lay.bits);
    if (a.cu || a.T == 0) pl.out = out;
    const int64_t items = std::max((a.cu ? (a.T + kBitRows - 1) / kBitRows : 0) + (pl.out ? a.nseq * 64 : 0), pl.nwords / 4);
    if (!many && !pl.bits && !pl.out) return hipSuccess;
    const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((items + 255) / 256, 1), 2048);
    hipLaunchKernelGGL(gated_plan_kernel, dim3(grid), dim3(256), 0, stream, a, pl);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_forward(GatedArgs a, const GatedLayout& lay, char* ws, hipStream_t stream) {
    GatedPass ps;
    const hipError_t e = run_plan(a, lay, ws, a.init, a.final_state, &ps, stream);
    if (e != hipSuccess || a.T == 0) return e;
    hipLaunchKernelGGL((gated_forward_kernel<T, Y>), dim3((unsigned)pass_blocks(ps)),
                       dim3(kFwdTile / kFwdRows * kSegLanes), 0, stream, a, ps);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_backward(GatedArgs a, const GatedLayout& lay, char* ws, hipStream_t stream) {
    GatedPass ps;
    hipError_t e = run_plan(a, lay, ws, a.dfinal, a.dinit, &ps, stream);
    if (e != hipSuccess) return e;
    float* part = (float*)(ws + lay.dlam);
    if (a.T > 0) {
        hipLaunchKernelGGL((gated_backward_kernel<T, Y>), dim3((unsigned)pass_blocks(ps)),
                           dim3(kBwdTile / kBwdRows * kSegLanes), 0, stream, a, ps, part);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(gated_dlam_kernel, dim3((unsigned)blocks_of(a.C, kSumCols)), dim3(kSumThreads), 0, stream, a, lay.ntiles,
                       (const float*)part, a.dlam);
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_gated_step(const GatedArgs& a, const float* state, float* state_out, hipStream_t stream) {
    const int64_t n = a.nseq * (a.C / kLaneCh);
    if (n == 0) return hipSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>(blocks_of(n, 256), 1 << 22);
    hipLaunchKernelGGL((gated_step_kernel<T, Y>), dim3(blocks), dim3(256), 0, stream, a, state, state_out);
    return hipGetLastError();
}

}  // namespace

GatedLayout gated_layout(int64_t T, int32_t C, bool packed, bool backward) {
    GatedLayout l;
    const int rows = backward ? kBwdTile : kFwdTile;
    l.ntiles = (T + rows - 1) / rows;
    l.ngroups = (l.ntiles + kGroup - 1) / kGroup;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const bool many = l.ntiles > 1;
    l.bits = take(packed ? (size_t)((T + kBitRows - 1) / kBitRows) * 4 : 0);
    l.maps = take(many ? (size_t)(l.ntiles + l.ngroups) * C * 8 : 0);
    l.counters = take(many ? (size_t)((C + kTileCh - 1) / kTileCh) * kGatedCounterStride * 4 : 0);
    l.dlam = take(backward ? (size_t)l.ntiles * C * 4 : 0);
    l.total = at;
    l.blocks = l.ntiles * ((C + kTileCh - 1) / kTileCh);
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
