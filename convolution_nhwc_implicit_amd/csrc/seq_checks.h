// seq_checks.h -- argument checks and small host helpers shared by the sequence
// operators' C entry points (seq_api.cpp, block_api.cpp).
#pragma once

#include <algorithm>

#include "seq_internal.h"

namespace cnv {

constexpr long long kMaxRows = (1LL << 31) - 1;
constexpr long long kMaxStride = (1LL << 24) - 1;  // 16 rows of it in bytes fit 31 bits
constexpr long long kMaxGridY = 65535;
constexpr int kCUs = 256;  // MI355X

inline bool float_type(int dtype) { return dtype == CONV2D_DTYPE_F16 || dtype == CONV2D_DTYPE_BF16 || dtype == CONV2D_DTYPE_F32; }
inline int bytes_of(int dtype) { return dtype == CONV2D_DTYPE_F32 ? 4 : 2; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t up(size_t v) { return (v + 255) / 256 * 256; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline int status(hipError_t e) { return e == hipSuccess ? CONV2D_OK : CONV2D_ERR_DEVICE; }

inline int check_batch(const seq_batch_t &b)
{
    if (b.seqs < 1 || b.len < 0 || b.tokens < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    if (!b.seq_start && b.tokens != (long long)b.seqs * b.len) return CONV2D_ERR_INVALID_ARGUMENT;
    if (b.tokens > kMaxRows || b.seqs > (1 << 24)) return CONV2D_ERR_UNSUPPORTED;
    return aligned(b.seq_start, 4) ? CONV2D_OK : CONV2D_ERR_UNSUPPORTED;
}

inline Seqs seqs_of(const seq_batch_t &b) { return Seqs{b.seq_start, b.seqs, b.len, b.tokens}; }
inline RowStride stride_of(const seq_stride_t &s) { return RowStride{s.row, s.seq}; }

inline bool all_aligned(size_t a, std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (!aligned(p, a)) return false;
    return true;
}

inline int lanes_for(int d, int v)
{
    int lanes = 1;
    while (lanes < 64 && (long long)lanes * v < d) lanes *= 2;
    return lanes;
}

inline int check_stride(const seq_stride_t &s)
{
    if (s.row < 0 || s.seq < 0) return CONV2D_ERR_INVALID_ARGUMENT;
    return s.row > kMaxStride ? CONV2D_ERR_UNSUPPORTED : CONV2D_OK;
}

// Cuts a workspace into pieces.
struct Carver {
    char *p;
    float *take(size_t bytes)
    {
        float *r = (float *)p;
        p += bytes;
        return r;
    }
};

}  // namespace cnv
