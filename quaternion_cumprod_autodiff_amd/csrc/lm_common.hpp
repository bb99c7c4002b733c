// lm_common.hpp -- what the gated-delta and query/key-norm kernels share:
// storage types, loads of several elements, host-side argument checks.  Not
// installed.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace qc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Storage types by dtype code (GDR_*, QKN_*).
template <int DT> struct Storage;
template <> struct Storage<0> { using type = float; };
template <> struct Storage<1> { using type = __bf16; };
template <> struct Storage<2> { using type = _Float16; };

constexpr size_t dtype_bytes(int dt) { return dt == 0 ? 4 : 2; }

// W consecutive elements as floats.  W elements of E are read as vectors of up
// to 16 bytes: the address must be aligned to min(16, W * sizeof(E)).
template <int W, class E>
__device__ __forceinline__ void load_floats(const E* p, float (&x)[W]) {
    constexpr int kPer = sizeof(E) * W >= 16 ? 16 / sizeof(E) : W;
    typedef E Vec __attribute__((ext_vector_type(kPer)));
    if constexpr (W == 1) {
        x[0] = float(p[0]);
    } else {
#pragma unroll
        for (int i = 0; i < W / kPer; ++i) {
            const Vec v = reinterpret_cast<const Vec*>(p)[i];
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[i * kPer + j] = float(v[j]);
        }
    }
}

// The reverse, each element rounded to nearest even once.
template <int W, class E>
__device__ __forceinline__ void store_floats(E* p, const float (&x)[W]) {
    constexpr int kPer = sizeof(E) * W >= 16 ? 16 / sizeof(E) : W;
    typedef E Vec __attribute__((ext_vector_type(kPer)));
    if constexpr (W == 1) {
        p[0] = E(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < W / kPer; ++i) {
            Vec v;
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = E(x[i * kPer + j]);
            reinterpret_cast<Vec*>(p)[i] = v;
        }
    }
}

// Host checks -----------------------------------------------------------------

struct ByteSpan {
    const void* p;
    size_t n;
};

inline bool spans_overlap(ByteSpan x, ByteSpan y) {
    if (!x.p || !y.p || !x.n || !y.n) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a < b + y.n && b < a + x.n;
}

// The first n_out spans are outputs: each must miss every other span.
inline bool outputs_overlap(const ByteSpan* s, int n_out, int n) {
    for (int i = 0; i < n_out; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && spans_overlap(s[i], s[j])) return true;
    return false;
}

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr int64_t kMaxElements = int64_t(1) << 40;

// a * b, or -1 where a factor is negative or the product passes kMaxElements.
inline int64_t count(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (a && b > kMaxElements / a) return -1;
    return a * b;
}

// Bytes from the first to behind the last element of [B, T, H, W] read
// through batch, token and head strides; -1 if a stride is negative or the
// extent passes the limit, 0 for an empty tensor.
inline int64_t strided_bytes(int64_t B, int64_t T, int64_t H, int64_t W, const int64_t st[3], size_t elem) {
    if (!B || !T || !H || !W) return 0;
    int64_t n = W;
    const int64_t size[3] = {B, T, H};
    for (int i = 0; i < 3; ++i) {
        const int64_t c = count(size[i] - 1, st[i]);
        if (c < 0) return -1;
        n += c;
    }
    return n > kMaxElements ? -1 : n * int64_t(elem);
}

// Whether rows of [.., W] read through these strides start on 16 bytes.
inline bool rows_on_16(const void* p, const int64_t st[3], size_t elem) {
    return aligned_to(p, 16) && st[0] * elem % 16 == 0 && st[1] * elem % 16 == 0 && st[2] * elem % 16 == 0;
}

}  // namespace qc
