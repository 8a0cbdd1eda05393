// Argument checks shared by the block operators' entry points: everything is
// refused on the host, before any launch.
#pragma once

#include <math.h>

#include "ssd.h"
#include "ssd_internal.h"

#define SSD_API extern "C" __attribute__((visibility("default")))
#define FAIL(st, ...) return (ssd_status)ssd::set_error_detail(st, __VA_ARGS__)

namespace ssd_checks {

constexpr int32_t kMaxChannels = 1 << 20;
constexpr int64_t kMaxBatch = 1 << 24;
constexpr int64_t kMaxElements = (int64_t)1 << 40;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

inline ssd_status ok() { return (ssd_status)ssd::set_error_detail(SSD_OK, "%s", ""); }

inline ssd_status queued(hipError_t e) {
    if (e != hipSuccess) FAIL(SSD_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

// A tensor argument: whether a NULL is an error, whether the call writes it, and
// its alignment.
struct Arg {
    const void* p;
    const char* name;
    bool required;
    bool output;
    unsigned align = 16;
};

// One output that may be the same tensor as some inputs (bits of their places
// in the list of arguments); no other output may.
struct InPlace {
    int output;
    uint32_t inputs;
};

// NULLs, alignment, and outputs that are an input or another output.
inline ssd_status check_args(const Arg* args, int n, InPlace in_place = {-1, 0}) {
    for (int i = 0; i < n; ++i) {
        if (!args[i].p) {
            if (args[i].required) FAIL(SSD_ERR_NULL, "%s is NULL", args[i].name);
            continue;
        }
        if ((uintptr_t)args[i].p & (args[i].align - 1u))
            FAIL(SSD_ERR_ALIGN, "%s is not %u-byte aligned", args[i].name, args[i].align);
    }
    for (int i = 0; i < n; ++i) {
        if (!args[i].p || !args[i].output) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || args[j].p != args[i].p || (i == in_place.output && in_place.inputs >> j & 1)) continue;
            FAIL(SSD_ERR_SHAPE, "%s aliases %s", args[i].name, args[j].name);
        }
    }
    return SSD_OK;
}

inline ssd_status check_dtypes(int32_t a, int32_t b) {
    if (a != SSD_F32 && a != SSD_BF16) FAIL(SSD_ERR_DTYPE, "dtype %d is neither SSD_F32 (0) nor SSD_BF16 (1)", a);
    if (b != SSD_F32 && b != SSD_BF16)
        FAIL(SSD_ERR_DTYPE, "the second dtype %d is neither SSD_F32 (0) nor SSD_BF16 (1)", b);
    return SSD_OK;
}

inline ssd_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need && !ws) FAIL(SSD_ERR_WORKSPACE, "workspace is NULL, %zu bytes are needed", need);
    if (have < need) FAIL(SSD_ERR_WORKSPACE, "workspace holds %zu bytes, %zu are needed", have, need);
    if ((uintptr_t)ws & 15u) FAIL(SSD_ERR_ALIGN, "workspace is not 16-byte aligned");
    return SSD_OK;
}

// Sizes and offsets shared by the sequence operators; fills *rows.
inline ssd_status check_sequences(int64_t batch, int64_t seqlen, int32_t channels, const int32_t* cu,
                           const int32_t* cu_host, int64_t* rows) {
    if (channels < 8 || channels > kMaxChannels || channels % 8 != 0)
        FAIL(SSD_ERR_SHAPE, "channels %d must be a multiple of 8 in [8, 2^20]", channels);
    if (batch < 0 || batch > kMaxBatch) FAIL(SSD_ERR_SHAPE, "batch must be in [0, 2^24]");
    if (seqlen < 0 || seqlen > kMaxRows) FAIL(SSD_ERR_SHAPE, "seqlen must be in [0, 2^31 - 1]");
    *rows = cu ? seqlen : batch * seqlen;  // < 2^55
    if (*rows > kMaxRows || *rows * channels > kMaxElements || batch * channels > kMaxElements)
        FAIL(SSD_ERR_SHAPE, "tensor too large");
    if (!cu && cu_host) FAIL(SSD_ERR_SHAPE, "cu_seqlens_host given without the device cu_seqlens");
    if (cu && batch == 0 && *rows > 0) FAIL(SSD_ERR_SHAPE, "packed rows without sequences");
    if (cu_host) {
        if (cu_host[0] != 0) FAIL(SSD_ERR_SEQLENS, "cu_seqlens[0] must be 0 (got %d)", cu_host[0]);
        for (int64_t s = 0; s < batch; ++s)
            if (cu_host[s + 1] < cu_host[s]) FAIL(SSD_ERR_SEQLENS, "cu_seqlens decreases at %lld", (long long)s);
        if (cu_host[batch] > *rows)
            FAIL(SSD_ERR_SEQLENS, "cu_seqlens[batch] = %d lies behind seqlen %lld", cu_host[batch], (long long)*rows);
    }
    return SSD_OK;
}

// A row stride in elements, 0 for dense.
inline ssd_status check_stride(const char* name, int64_t stride, int32_t width, int64_t rows, int64_t* out) {
    *out = stride ? stride : width;
    if (stride < 0 || *out < width || *out % 8 != 0)
        FAIL(SSD_ERR_SHAPE, "%s %lld must be 0 or a multiple of 8 of at least %d", name, (long long)stride, width);
    if (rows > 0 && *out > kMaxElements / rows) FAIL(SSD_ERR_SHAPE, "%s: tensor too large", name);
    return SSD_OK;
}

}  // namespace ssd_checks
