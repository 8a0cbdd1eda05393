// Which rows of a dense or packed batch belong to which sequence, and where
// sequences begin and end inside a run of rows: whole numbers only, so that
// the host can compute it too.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define SSD_HOST_DEVICE __host__ __device__
#else
#define SSD_HOST_DEVICE
#endif

namespace ssd {

SSD_HOST_DEVICE inline int64_t clamp_row(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// Offsets are clamped into [0, T] with the end no earlier than the start, so
// no row or state index derived from them leaves its array, whatever the
// device list holds.
struct RowRange {
    int64_t lo, hi;
};

SSD_HOST_DEVICE inline RowRange seq_range(const int32_t* cu, int64_t L, int64_t T, int64_t s) {
    if (!cu) return {s * L, s * L + L};
    const int64_t lo = clamp_row(cu[s], 0, T);
    return {lo, clamp_row(cu[s + 1], lo, T)};
}

// Rows that belong to sequences.  Rows outside (behind the last sequence) are
// neither read into a result nor written.
SSD_HOST_DEVICE inline RowRange live_rows(const int32_t* cu, int64_t nseq, int64_t T) {
    if (!cu) return {0, T};
    const int64_t lo = clamp_row(cu[0], 0, T);
    return {lo, clamp_row(cu[nseq], lo, T)};
}

// The sequence holding a live row: the last one that starts at or before it.
SSD_HOST_DEVICE inline int64_t seq_of(const int32_t* cu, int64_t nseq, int64_t L, int64_t row) {
    if (!cu) return (uint32_t)row / (uint32_t)L;  // rows < 2^31
    int64_t lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------- boundaries
// A word of boundary bits: bit j: row t0 + j is its sequence's first one; bit
// 16 + j: its last one.
constexpr int kBitRows = 8;  // rows per word of a packed batch

// Packed: the word of the kBitRows rows from t0.  Every offset in [t0, t1] ends
// a sequence at the row before it and starts one at its row.
SSD_HOST_DEVICE inline uint32_t packed_boundaries(const int32_t* cu, int64_t nseq, RowRange live, int64_t t0) {
    const int64_t t1 = t0 + kBitRows < live.hi ? t0 + kBitRows : live.hi;
    uint32_t m = 0;
    for (int64_t t = t0 > live.lo ? t0 : live.lo; t <= t1;) {
        int64_t lo = 0, hi = nseq;  // the first offset >= t
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (cu[mid] < t) lo = mid + 1;
            else hi = mid;
        }
        const int64_t at = cu[lo] > t ? cu[lo] : t;
        if (at > t1) break;
        if (at < t1) m |= 1u << (at - t0);
        if (at > t0) m |= 1u << (15 + at - t0);
        t = at + 1;
    }
    return m;
}

// Dense: the word of ROWS rows from t0.
template <int ROWS>
SSD_HOST_DEVICE inline uint32_t dense_boundaries(int64_t L, int64_t t0) {
    uint32_t m = 0;
    const uint32_t p = (uint32_t)t0 % (uint32_t)L;  // rows < 2^31
    for (int64_t j = p ? L - p : 0; j <= ROWS; j += L) {
        if (j < ROWS) m |= 1u << j;
        if (j > 0) m |= 1u << (15 + j);
    }
    return m;
}

// The boundary bits of ROWS rows from t0 (a multiple of ROWS), and which of them
// are live (bit j).  words: of packed_boundaries.  A row that is not live has no
// boundary: a dense batch goes on past its last row in dense_boundaries, to
// sequences that have no initial state to be read.
struct RunBits {
    uint32_t bits, live;
};

template <int ROWS>
SSD_HOST_DEVICE inline RunBits run_bits(const int32_t* cu, const uint32_t* words, int64_t nseq, int64_t L, int64_t T,
                                        int64_t t0) {
    static_assert(kBitRows % ROWS == 0, "a run lies in one word");
    RunBits r{0, 0};
    if (t0 >= T) return r;
    if (cu) r.bits = words[t0 / kBitRows] >> (t0 % kBitRows) & (((1u << ROWS) - 1) * 0x10001u);
    else r.bits = dense_boundaries<ROWS>(L, t0);
    const RowRange rows = live_rows(cu, nseq, T);
    const int lo = (int)clamp_row(rows.lo - t0, 0, ROWS), hi = (int)clamp_row(rows.hi - t0, lo, ROWS);
    r.live = ((1u << hi) - 1) & ~((1u << lo) - 1);
    r.bits &= r.live | r.live << 16;
    return r;
}

}  // namespace ssd
