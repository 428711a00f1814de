// seq_common.h -- element types, sequence geometry and small device helpers
// of the sequence operators (causal convolution, selective scan, fp8 products).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "device_common.h"
#include "sequence_ops.h"

namespace cnv {

// ---- element types: storage, and conversion to and from fp32 ----------------
struct SF16 {
    using S = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static inline float to(S e) { return f16_to_f32(e); }
    __device__ static inline S from(float v) { return f32_to_f16(v); }
};
struct SBF16 {
    using S = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static inline float to(S e) { return bf16_to_f32(e); }
    __device__ static inline S from(float v) { return f32_to_bf16(v); }
};
struct SF32 {
    using S = float;
    static constexpr int kBytes = 4;
    __device__ static inline float to(S e) { return e; }
    __device__ static inline S from(float v) { return v; }
};

// V elements moved by one load or store.  Tensors are only aligned to their
// element (odd channel counts, sliced projections); global memory takes wide
// accesses at any address, so the type says so and the compiler keeps them wide.
template <class S, int V>
struct __attribute__((packed, aligned(sizeof(S)))) SVec {
    S v[V];
};

template <class E, int V>
__device__ inline void load_vec(const typename E::S *p, int have, float (&out)[V])
{
    if (have >= V) {
        const SVec<typename E::S, V> r = *(const SVec<typename E::S, V> *)p;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = E::to(r.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = i < have ? E::to(p[i]) : 0.0f;
    }
}

template <class E, int V>
__device__ inline void store_vec(typename E::S *p, int have, const float (&in)[V])
{
    if (have >= V) {
        SVec<typename E::S, V> r;
#pragma unroll
        for (int i = 0; i < V; ++i) r.v[i] = E::from(in[i]);
        *(SVec<typename E::S, V> *)p = r;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < have) p[i] = E::from(in[i]);
    }
}

// A value that every lane of the wave holds, in a scalar register.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- sequences ---------------------------------------------------------------
// `tokens` rows hold `seqs` sequences: [seqs][len] when start is null, else
// sequence s is rows start[s] .. start[s+1]-1.  start is device memory that the
// host cannot check, so every value is clamped to the rows that exist.
struct Seqs {
    const int *start;
    int seqs, len;
    long long tokens;
    __device__ inline long long begin(int s) const
    {
        if (!start) return (long long)s * len;
        const long long v = start[s];
        return v < 0 ? 0 : (v > tokens ? tokens : v);
    }
    __device__ inline long long end(int s) const  // never before begin(s)
    {
        const long long b = begin(s), e = begin(s + 1);
        return e < b ? b : e;
    }
    // the last sequence that starts at or before row t (0 if none does)
    __device__ inline int find(long long t) const
    {
        if (!start) return (int)(t / len);
        int lo = 0, hi = seqs;  // begin(lo) <= t < begin(hi), were start sorted
        while (hi - lo > 1) {
            const int m = lo + (hi - lo) / 2;
            if (begin(m) <= t) lo = m; else hi = m;
        }
        return lo;
    }
};

// Strides, in elements, of a tensor of rows: between rows, and between the
// sequences of a dense batch.
struct RowStride {
    long long row, seq;
    __device__ inline long long at(const Seqs &q, int s, long long t) const
    {
        return q.start ? t * row : s * seq + (t - (long long)s * q.len) * row;
    }
};

// ---- activations ---------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// 1 / (1 + e^-v); e^-v past the largest float gives 0
__device__ inline float sigmoid_f32(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}

}  // namespace cnv
